// kv8_append.cu -- page2d rotary embedding of new tokens and their append to a cache held in
// e4m3 with one scale per (page, head).
//
// The same rotation and the same cache rows as the bf16 form (rope_append.cu; Unlimited-OCR-2
// walk-through, news.rkmt.cn/news/25027, sections 四 and 六).  The tokens of one sequence are
// appended together, so that a page's scale is decided once per call.  For the rows that a call
// adds to a (page, head), separately for K and V:
//   need = 2^max(ceil(log2(amax / 448)), -126),  amax over the rows' finite values;
//   s    = need when the page holds no older row of the sequence,
//          max(s_old rounded up to a power of two, need) otherwise;
//   new code = e4m3(x / s), older code c -> e4m3(c s_old / s).
// A scale is a power of two, so that dividing by it is exact, and raising it moves the older codes'
// exponents: they are rounded again only where they fall below e4m3's normal range.  It only
// rises, and rows that are already cached keep their codes unless it does.
//
// x is the rotated key in 64 bits (angles, sines and products) rounded once, to nearest even: on
// its way through 32 bits it is rounded to odd, which no later rounding to fewer bits can see.  So
// a code is a function of its inputs' exact values, the same whatever chunk its token came in.
// Infinities and NaN are stored as e4m3's NaN (it has no infinity, and a saturated one would look
// like a value).
//
// Layout: CTA (run, head), a run being the new tokens of one sequence that fall in one page; head
// index H stands for the indexer's vectors, which stay bf16.
#include <math.h>

#include "kernels.h"
#include "kv8.cuh"

namespace uocr {

namespace {
constexpr int kPairs = kD / 2;
constexpr int kAppThreads = 128;
constexpr int kMinExp = -126;   // the least scale: 2^-126, the smallest normal fp32

// x rounded to fp32 to odd: an exact x stays, any other gets the neighbour whose last bit is 1.
__device__ __forceinline__ float round_odd(double x) {
    const float t = __double2float_rz(x);
    return (double)t != x && isfinite(t) ? __uint_as_float(__float_as_uint(t) | 1u) : t;
}

// Exponent e of the least power of two with 2 half <= 448 * 2^e, at least kMinExp.  half >= 0, finite.
__device__ __forceinline__ int scale_exp(float half) {
    const uint32_t b = __float_as_uint(half);
    const int e = (int)(b >> 23) - 127;
    // half = m 2^e with m in [1, 2): 448 = 1.75 * 2^8
    return max(kMinExp, (b & 0x7fffffu) <= 0x600000u ? e - 7 : e - 6);
}

// A stored scale rounded up to a power of two: its exponent, in [kMinExp, 127].
__device__ __forceinline__ int scale_exp_of(float s) {
    const uint32_t b = __float_as_uint(s);
    if (!(s >= 1.17549435e-38f)) return kMinExp;   // not positive, subnormal or NaN
    const int e = (int)(b >> 23) - 127 + ((b & 0x7fffffu) ? 1 : 0);
    return min(e, 127);
}

__device__ __forceinline__ float exp2i(int e) {   // 2^e, e in [-127, 127]
    return e > -127 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x400000u);
}

__device__ __forceinline__ uint8_t to_e4m3(float x) {
    if (!isfinite(x)) return 0x7f;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return (uint8_t)(r & 0xff);
}

__device__ __forceinline__ float from_e4m3(uint8_t c) {
    const uint32_t h = e4m3x2_to_f16x2((uint16_t)c);
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

// A run: the new tokens first .. first + count - 1 of sequence b, at rows row .. of logical block lp.
struct Run {
    int b, first, count, lp, row;
};

// Run r of the call, or false.  Sequence b's runs start at slot start[b] / 32 + 2 b: it needs at
// most count / 32 + 2 of them, and slots of later sequences begin past those.
__device__ __forceinline__ bool find_run(int r, const int32_t *__restrict__ start,
                                         const int32_t *__restrict__ seq_lens, int n, int B, int max_blocks,
                                         int32_t *dev_err, bool report, Run &run) {
    int b, a, e, slot;
    if (start) {
        int lo = 0, hi = B;   // the last sequence whose first slot is at most r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((long long)__ldg(start + mid) / kBlock + 2ll * mid <= r)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        a = __ldg(start + b);
        e = __ldg(start + b + 1);
        if (a < 0 || e < a || e > n) {
            if (report) flag_error(dev_err, UOCR_DEVERR_POS);
            return false;
        }
        slot = r - (a / kBlock + 2 * b);
        if (slot < 0) return false;
    } else {
        b = a = r;
        e = r + 1;
        slot = 0;
    }
    if (a == e) return false;
    const int len = __ldg(seq_lens + b);
    if (len < e - a || len > max_blocks * kBlock) {
        if (report) flag_error(dev_err, UOCR_DEVERR_POS);
        return false;
    }
    const int base = len - (e - a);   // position of the sequence's first new token
    const int lp = base / kBlock + slot;
    if (lp > (len - 1) / kBlock) return false;
    const int p0 = max(lp * kBlock, base), p1 = min(len, (lp + 1) * kBlock);
    run = {b, a + (p0 - base), p1 - p0, lp, p0 - lp * kBlock};
    return true;
}
}  // namespace

__global__ void __launch_bounds__(kAppThreads)
rope_append_kv8_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *idx_q, const __nv_bfloat16 *__restrict__ k_new,
                       const __nv_bfloat16 *__restrict__ v_new, const __nv_bfloat16 *__restrict__ idx_k_new,
                       const int32_t *__restrict__ tok_pos, const int32_t *__restrict__ page_pos,
                       const int32_t *__restrict__ start, const int32_t *__restrict__ bt,
                       const int32_t *__restrict__ seq_lens, int n, int B, int H, int max_blocks, int num_pages,
                       __nv_bfloat16 *q_out, __nv_bfloat16 *idx_q_out, uint8_t *__restrict__ k_cache,
                       uint8_t *__restrict__ v_cache, float *__restrict__ k_scale, float *__restrict__ v_scale,
                       __nv_bfloat16 *__restrict__ idx_k_cache, RopeFreqs freqs, int32_t *dev_err) {
    // half of the run's rotated keys (a rotation of bf16's largest numbers leaves fp32), rounded to
    // odd; then half of its values
    __shared__ float s_x[kBlock][kD];
    __shared__ float s_red[kAppThreads / 32];
    const int h = blockIdx.y, tid = threadIdx.x;
    Run run;
    if (!find_run(blockIdx.x, start, seq_lens, n, B, max_blocks, dev_err, tid == 0 && h == 0, run)) return;
    int page = __ldg(bt + (size_t)run.b * max_blocks + run.lp);
    if ((unsigned)page >= (unsigned)num_pages) {
        if (tid == 0 && h == 0) flag_error(dev_err, UOCR_DEVERR_PAGE);
        page = -1;
    }

    // rotate: thread (x, pair) takes tokens x, x + 2, ..
    const int pair = tid & (kPairs - 1);
    float amax = 0.f;
    for (int t = tid / kPairs; t < run.count; t += kAppThreads / kPairs) {
        const int i = run.first + t;
        const int page_mod2 = ((__ldg(page_pos + i) % 2) + 2) % 2;
        const double coord = pair < kPairs - UOCR_ROPE_PAGE_PAIRS ? (double)__ldg(tok_pos + i) : (double)page_mod2;
        double sn, cs;
        sincos(coord * freqs.inv[pair], &sn, &cs);
        const __nv_bfloat16 *src = h < H ? q + ((size_t)i * H + h) * kD : idx_q + (size_t)i * kDIdx;
        __nv_bfloat16 *dst = h < H ? q_out + ((size_t)i * H + h) * kD : idx_q_out + (size_t)i * kDIdx;
        double x0 = (double)__bfloat162float(src[pair]), x1 = (double)__bfloat162float(src[pair + kPairs]);
        dst[pair] = __float2bfloat16_rn(round_odd(x0 * cs - x1 * sn));
        dst[pair + kPairs] = __float2bfloat16_rn(round_odd(x1 * cs + x0 * sn));
        src = h < H ? k_new + ((size_t)i * H + h) * kD : idx_k_new + (size_t)i * kDIdx;
        x0 = (double)__bfloat162float(src[pair]);
        x1 = (double)__bfloat162float(src[pair + kPairs]);
        const double r0 = x0 * cs - x1 * sn, r1 = x1 * cs + x0 * sn;
        if (h < H) {
            const float y0 = round_odd(0.5 * r0), y1 = round_odd(0.5 * r1);
            s_x[t][pair] = y0;
            s_x[t][pair + kPairs] = y1;
            if (isfinite(y0)) amax = fmaxf(amax, fabsf(y0));
            if (isfinite(y1)) amax = fmaxf(amax, fabsf(y1));
        } else if (page >= 0) {
            __nv_bfloat16 *row = idx_k_cache + ((size_t)page * kBlock + run.row + t) * kDIdx;
            row[pair] = __float2bfloat16_rn(round_odd(r0));
            row[pair + kPairs] = __float2bfloat16_rn(round_odd(r1));
        }
    }
    if (h == H || page < 0) return;

    const size_t tile = (size_t)page * H + h;
    for (int which = 0; which < 2; ++which) {
        uint8_t *codes = (which ? v_cache : k_cache) + tile * kTile8;
        float *scale = (which ? v_scale : k_scale) + tile;
        if (which) {
            __syncthreads();   // the keys are read
            amax = 0.f;
            for (int x = tid; x < run.count * kD; x += kAppThreads) {
                const float y = 0.5f * __bfloat162float(v_new[((size_t)(run.first + x / kD) * H + h) * kD + x % kD]);
                s_x[x / kD][x % kD] = y;
                if (isfinite(y)) amax = fmaxf(amax, fabsf(y));
            }
        }
        amax = warp_max(amax);
        if ((tid & 31) == 0) s_red[tid >> 5] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
        int e = scale_exp(amax);
        if (run.row > 0) {
            const float old = *scale;
            e = max(e, scale_exp_of(old));
            const float ratio = old / exp2i(e);
            if (ratio != 1.f)
                for (int x = tid; x < run.row * kD; x += kAppThreads) codes[x] = to_e4m3(from_e4m3(codes[x]) * ratio);
        }
        const float inv = exp2i(1 - e);
        for (int x = tid; x < run.count * kD; x += kAppThreads)
            codes[run.row * kD + x] = to_e4m3(s_x[x / kD][x % kD] * inv);
        __syncthreads();   // every thread has read the old scale and s_red
        if (tid == 0) *scale = exp2i(e);
    }
}

cudaError_t launch_rope_append_kv8(const LaunchCtx &c, const void *q, const void *idx_q, const void *k_new,
                                   const void *v_new, const void *idx_k_new, const int32_t *tok_pos,
                                   const int32_t *page_pos, const int32_t *start, const int32_t *bt,
                                   const int32_t *seq_lens, int n, int B, int H, int max_blocks, int num_pages,
                                   void *q_out, void *idx_q_out, void *k_cache, void *v_cache, float *k_scale,
                                   float *v_scale, void *idx_k_cache, int32_t *dev_err) {
    const long long runs = start ? (long long)n / kBlock + 2ll * B : n;
    if (runs > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    rope_append_kv8_kernel<<<dim3((unsigned)runs, (unsigned)(H + 1)), kAppThreads, 0, c.stream>>>(
        (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)idx_q, (const __nv_bfloat16 *)k_new,
        (const __nv_bfloat16 *)v_new, (const __nv_bfloat16 *)idx_k_new, tok_pos, page_pos, start, bt, seq_lens, n, B, H,
        max_blocks, num_pages, (__nv_bfloat16 *)q_out, (__nv_bfloat16 *)idx_q_out, (uint8_t *)k_cache,
        (uint8_t *)v_cache, k_scale, v_scale, (__nv_bfloat16 *)idx_k_cache, rope_freqs(), dev_err);
    return cudaGetLastError();
}

}  // namespace uocr
