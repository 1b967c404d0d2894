// kv8_append.cu -- page2d rotary embedding of new tokens and their append to a cache held in
// e4m3 with one scale per (page, head).
//
// The same rotation and the same cache rows as the bf16 form (rope_append.cu; Unlimited-OCR-2
// walk-through, news.rkmt.cn/news/25027, sections 四 and 六).  The tokens of one sequence are
// appended together, so that a page's scale is decided once per call.  For the rows that a call
// adds to a (page, head), separately for K and V:
//   need = 2^max(ceil(log2(amax / 448)), -126),  amax over the rows' finite values;
//   s    = need when the page holds no older row of the sequence,
//          max(|s_old| rounded up to a power of two, need) otherwise;
//   new code = e4m3(x / s), older code c -> e4m3(c s_old / s).
// A scale is a power of two, so that dividing by it is exact, and raising it moves the older codes'
// exponents: they are rounded again only where they fall below e4m3's normal range.  It only
// rises, and rows that are already cached keep their codes unless it does.
//
// x is the rotated key in 64 bits (angles, sines; products in 64 bits or as sums of two fp32
// numbers) rounded once, to nearest even: on its way through 32 bits it is rounded to odd, which no
// later rounding to fewer bits can see.  So
// a code is a function of its inputs' exact values, the same whatever chunk its token came in.  The
// rotated queries and indexer vectors are rounded once to bf16 in the same way, so that neither
// they nor the blocks that they select depend on the chunk.
// Infinities and NaN are stored as e4m3's NaN (it has no infinity, and a saturated one would look
// like a value).
//
// Layout: a run is the new tokens of one sequence that fall in one page; head index H stands for the
// indexer's vectors, which stay bf16.  Two kernels:
//   few tokens a sequence (decode): CTA (run, head), a thread per (token, pair); what counts is the
//       latency of one sine and one reduction.  64 sequences of one token, 10 heads: 4.4 us.
//   many: CTA (run, a few heads), thread (token, 8 pairs) of 32 tokens: the sines of a page are
//       formed once for the CTA's heads and kept in registers, every load and store is 8 or 16 bytes.
//       2048 tokens, 10 heads: 27.7 us with the first kernel (11 times the sines, 64-bit conversions
//       at 16 a clock), 15.4 here: bound by the issue of the rotation's two-number products (1260
//       instructions a warp and head, its share of the sines counted; 45 % of the issue slots) and one
//       barrier a head, not by its 28 MB (4.3 us).  1.5 of the 15.4 are what the queries' single rounding
//       costs (a test of each value in fp32).
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

// Pair (x0, x1) turned by an angle, in 64 bits.  (Spelled out, so that every kernel's products and sums
// are rounded alike.)
__device__ __forceinline__ void turn(double x0, double x1, double cs, double sn, double &r0, double &r1) {
    r0 = fma(x0, cs, -__dmul_rn(x1, sn));
    r1 = fma(x1, cs, __dmul_rn(x0, sn));
}

// Exponent e of the least power of two with 2 half <= 448 * 2^e, at least kMinExp.  half >= 0, finite.
__device__ __forceinline__ int scale_exp(float half) {
    const uint32_t b = __float_as_uint(half);
    const int e = (int)(b >> 23) - 127;
    // half = m 2^e with m in [1, 2): 448 = 1.75 * 2^8
    return max(kMinExp, (b & 0x7fffffu) <= 0x600000u ? e - 7 : e - 6);
}

// A stored scale's magnitude rounded up to a power of two: its exponent, in [kMinExp, 127].  (A negative
// scale turns its codes' signs when they are rescaled.)
__device__ __forceinline__ int scale_exp_of(float s) {
    const uint32_t b = __float_as_uint(fabsf(s));
    if (!(fabsf(s) >= 1.17549435e-38f)) return kMinExp;   // zero, subnormal or NaN
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

// code * ratio rounded to odd: a ratio that is not a power of two has 24 bits, and a product of 28
// rounded to fp32 first could reach a midpoint of e4m3 that it only lies beside.
__device__ __forceinline__ float rescaled(float code, float ratio) {
    const float p = __fmul_rz(code, ratio);
    return fmaf(code, ratio, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
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
    if (!start && len == 0) return false;   // an empty place of a padded batch has no new token
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
rope_append_kv8_few_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *idx_q, const __nv_bfloat16 *__restrict__ k_new,
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
        double r0, r1;
        turn((double)__bfloat162float(src[pair]), (double)__bfloat162float(src[pair + kPairs]), cs, sn, r0, r1);
        dst[pair] = __float2bfloat16_rn(round_odd(r0));
        dst[pair + kPairs] = __float2bfloat16_rn(round_odd(r1));
        src = h < H ? k_new + ((size_t)i * H + h) * kD : idx_k_new + (size_t)i * kDIdx;
        turn((double)__bfloat162float(src[pair]), (double)__bfloat162float(src[pair + kPairs]), cs, sn, r0, r1);
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
                for (int x = tid; x < run.row * kD; x += kAppThreads) codes[x] = to_e4m3(rescaled(from_e4m3(codes[x]), ratio));
        }
        const float inv = exp2i(1 - e);
        for (int x = tid; x < run.count * kD; x += kAppThreads)
            codes[run.row * kD + x] = to_e4m3(s_x[x / kD][x % kD] * inv);
        __syncthreads();   // every thread has read the old scale and s_red
        if (tid == 0) *scale = exp2i(e);
    }
}

namespace {
constexpr int kManyThreads = kBlock * kPairs / 8;   // thread (token, 8 pairs)

// hi + lo, rounded to odd.
__device__ __forceinline__ float round_odd(float hi, float lo) {
    if (lo == 0.f) return hi;   // (keeps the sign of a zero)
    const float s = __fadd_rz(hi, lo);
    return (hi - s) + lo != 0.f && isfinite(s) ? __uint_as_float(__float_as_uint(s) | 1u) : s;
}

// a x + b y to about 2^-46 of its terms, rounded to odd; a and b as sums of two fp32 numbers.  Products
// with their rounding errors by fma, the sum with its own by Knuth's TwoSum, and an odd rounding (Boldo and
// Melquiond: a later rounding to fewer bits then is the only one).  Written with the functions that are
// never joined: made one fma, p + q is no longer the sum of the two whose errors are added below, and the
// result is off by 2^-25.
__device__ __forceinline__ float dot2_odd(float x, float ah, float al, float y, float bh, float bl) {
    const float p = __fmul_rn(x, ah), pe = fmaf(x, ah, -p);
    const float q = __fmul_rn(y, bh), qe = fmaf(y, bh, -q);
    const float s = __fadd_rn(p, q), t = __fsub_rn(s, p);
    const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(q, t));
    return round_odd(s, fmaf(x, al, fmaf(y, bl, __fadd_rn(e, __fadd_rn(pe, qe)))));
}

// Eight numbers (times inv) to packed codes; what is not finite to NaN.
__device__ __forceinline__ uint2 pack_e4m3(const float *x, float inv) {
    uint16_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float nan = __uint_as_float(0x7fffffffu);
        const float a = isfinite(x[2 * k]) ? x[2 * k] * inv : nan, b = isfinite(x[2 * k + 1]) ? x[2 * k + 1] * inv : nan;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r[k]) : "f"(b), "f"(a));
    }
    return make_uint2((uint32_t)r[0] | (uint32_t)r[1] << 16, (uint32_t)r[2] | (uint32_t)r[3] << 16);
}

// 16 codes times ratio, to codes.
__device__ __forceinline__ uint4 rescale_e4m3(uint4 v, float ratio) {
    uint32_t out[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t lo, hi;
        e4m3x4_to_f16(word(v, w), lo, hi);
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        uint16_t r0, r1;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r0) : "f"(rescaled(a.y, ratio)), "f"(rescaled(a.x, ratio)));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r1) : "f"(rescaled(b.y, ratio)), "f"(rescaled(b.x, ratio)));
        out[w] = (uint32_t)r0 | (uint32_t)r1 << 16;
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Whether 64 bits that are off by up to `off` round to bf16 as their exact value does: they are not that
// near a midpoint.  False for what is below bf16's normal range or not finite.
__device__ __forceinline__ bool decided(double r, double off) {
    const double a = fabs(r);
    const long long midpoint = (__double_as_longlong(a) & ~((1ll << 45) - 1)) | 1ll << 44;
    return a >= 0x1p-126 && fabs(a - __longlong_as_double(midpoint)) > off;
}

// A pair turned and rounded to odd, as the few-token kernel does.  The sum of the two fp32 numbers that
// stand for a sine is off by 2^-49, which nearly always decides the rounding; else the sine is formed again.
__device__ __noinline__ float2 turn_exactly(float x0, float x1, float ch, float cl, float sh, float sl, int coord,
                                            double inv) {
    double r0, r1;
    turn((double)x0, (double)x1, (double)ch + (double)cl, (double)sh + (double)sl, r0, r1);
    const double off = (fabs((double)x0) + fabs((double)x1)) * 0x1p-44;
    if (!decided(r0, off) || !decided(r1, off)) {
        double sn, cs;
        sincos((double)coord * inv, &sn, &cs);
        turn((double)x0, (double)x1, cs, sn, r0, r1);
    }
    return make_float2(round_odd(r0), round_odd(r1));
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        r[k] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
}  // namespace

__global__ void __launch_bounds__(kManyThreads, 2)
rope_append_kv8_many_kernel(const uint4 *q, const uint4 *idx_q, const uint4 *__restrict__ k_new,
                            const uint4 *__restrict__ v_new, const uint4 *__restrict__ idx_k_new,
                            const int32_t *__restrict__ tok_pos, const int32_t *__restrict__ page_pos,
                            const int32_t *__restrict__ start, const int32_t *__restrict__ bt,
                            const int32_t *__restrict__ seq_lens, int n, int B, int H, int max_blocks,
                            int num_pages, int group, uint4 *q_out, uint4 *idx_q_out, uint8_t *__restrict__ k_cache,
                            uint8_t *__restrict__ v_cache, float *__restrict__ k_scale,
                            float *__restrict__ v_scale, uint4 *__restrict__ idx_k_cache, RopeFreqs freqs,
                            int32_t *dev_err) {
    constexpr int kWarps = kManyThreads / 32;
    __shared__ float2 s_red[2][kWarps];
    const int tid = threadIdx.x, t = tid >> 3, c = tid & 7;   // token of the run, pairs 8 c .. 8 c + 7
    const int h0 = blockIdx.y * group, h1 = min(H + 1, h0 + group);
    Run run;
    if (!find_run(blockIdx.x, start, seq_lens, n, B, max_blocks, dev_err, tid == 0 && h0 == 0, run)) return;
    int page = __ldg(bt + (size_t)run.b * max_blocks + run.lp);
    if ((unsigned)page >= (unsigned)num_pages) {
        if (tid == 0 && h0 == 0) flag_error(dev_err, UOCR_DEVERR_PAGE);
        page = -1;
    }
    const bool mine = t < run.count;
    const int i = run.first + (mine ? t : 0);
    auto coord = [&](int pair) {
        return pair < kPairs - UOCR_ROPE_PAGE_PAIRS ? __ldg(tok_pos + i) : ((__ldg(page_pos + i) % 2) + 2) % 2;
    };
    // cosines and sines of the thread's pairs, as sums of two fp32 numbers
    float ch[8], cl[8], sh[8], sl[8];
    if (mine) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            double sn, cs;
            sincos((double)coord(8 * c + e) * freqs.inv[8 * c + e], &sn, &cs);
            ch[e] = (float)cs;
            cl[e] = (float)(cs - (double)ch[e]);
            sh[e] = (float)sn;
            sl[e] = (float)(sn - (double)sh[e]);
        }
    }
    // Eight pairs to bf16, rounded once from their value in 64 bits as in the few-token kernel.  In fp32
    // a value is off by at most 2.5 * 2^-24 of its terms (a product's rounding, the sum's, half a unit of
    // each sine); only where that could take it over a midpoint of bf16 (some 2^-11 of all values), or a term
    // is not finite, is its pair turned in 64 bits.
    auto rotate_bf16 = [&](const uint4 (&in)[2], uint4 &low, uint4 &high) {
        float x0[8], x1[8], o0[8], o1[8];
        bf16x8_to_f32(in[0], x0);
        bf16x8_to_f32(in[1], x1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            o0[e] = fmaf(x0[e], ch[e], -x1[e] * sh[e]);
            o1[e] = fmaf(x1[e], ch[e], x0[e] * sh[e]);
            const float off = fmaf(fabsf(x0[e]) + fabsf(x1[e]), 0x1.8p-23f, 0x1p-146f);   // (fp32's least values too)
            auto far = [&](float o) {   // from the midpoint of its bf16 neighbours; false for NaN
                return fabsf(o - __uint_as_float((__float_as_uint(o) & 0xffff0000u) | 0x8000u)) > off;
            };
            if (!far(o0[e]) || !far(o1[e])) {
                const float2 o = turn_exactly(x0[e], x1[e], ch[e], cl[e], sh[e], sl[e], coord(8 * c + e), freqs.inv[8 * c + e]);
                o0[e] = o.x;
                o1[e] = o.y;
            }
        }
        low = pack_bf16x8(o0);
        high = pack_bf16x8(o1);
    };

    for (int h = h0; h < h1; ++h) {
        const bool idx = h == H;
        const size_t row = (idx ? (size_t)i : (size_t)i * H + h) * (kD / 8);
        uint4 qv[2], kv[2], vv[2];
        float2 old = make_float2(0.f, 0.f);
        const size_t tile = (size_t)max(page, 0) * H + (idx ? 0 : h);
        if (mine) {
            const uint4 *src = idx ? idx_q : q;
            qv[0] = src[row + c];
            qv[1] = src[row + 8 + c];
            src = idx ? idx_k_new : k_new;
            kv[0] = __ldg(src + row + c);
            kv[1] = __ldg(src + row + 8 + c);
            if (!idx) {
                vv[0] = __ldg(v_new + row + 2 * c);
                vv[1] = __ldg(v_new + row + 2 * c + 1);
            }
        }
        // read before any thread of the CTA writes the new ones
        if (!idx && run.row > 0 && page >= 0) old = make_float2(k_scale[tile], v_scale[tile]);

        float y[16], v[16];   // half of the rotated key (dims 8 c .. and 64 + 8 c ..), half of the values
        float2 top = make_float2(0.f, 0.f);
        if (mine) {
            uint4 low, high;
            rotate_bf16(qv, low, high);
            uint4 *dst = idx ? idx_q_out : q_out;
            dst[row + c] = low;
            dst[row + 8 + c] = high;
            if (idx) {
                rotate_bf16(kv, low, high);
                if (page >= 0) {
                    uint4 *to = idx_k_cache + ((size_t)page * kBlock + run.row + t) * (kDIdx / 8);
                    to[c] = low;
                    to[8 + c] = high;
                }
            } else {
                float x0[8], x1[8];
                bf16x8_to_f32(kv[0], x0);
                bf16x8_to_f32(kv[1], x1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = 0.5f * x0[e], b = 0.5f * x1[e];
                    y[e] = dot2_odd(a, ch[e], cl[e], -b, sh[e], sl[e]);
                    y[8 + e] = dot2_odd(b, ch[e], cl[e], a, sh[e], sl[e]);
                }
                float w[8];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    bf16x8_to_f32(vv[k], w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[8 * k + e] = 0.5f * w[e];
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (isfinite(y[e])) top.x = fmaxf(top.x, fabsf(y[e]));
                    if (isfinite(v[e])) top.y = fmaxf(top.y, fabsf(v[e]));
                }
            }
        }
        if (idx || page < 0) continue;   // uniform over the CTA
        top = make_float2(warp_max(top.x), warp_max(top.y));
        float2(&red)[kWarps] = s_red[h & 1];   // two in turn: one barrier a head
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
        float2 amax = red[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) amax = make_float2(fmaxf(amax.x, red[w].x), fmaxf(amax.y, red[w].y));
        int ek = scale_exp(amax.x), ev = scale_exp(amax.y);
        uint8_t *kt = k_cache + tile * kTile8, *vt = v_cache + tile * kTile8;
        if (run.row > 0) {
            ek = max(ek, scale_exp_of(old.x));
            ev = max(ev, scale_exp_of(old.y));
            const float rk = old.x / exp2i(ek), rv = old.y / exp2i(ev);
            if (t < run.row) {   // older row t, 16 codes
                uint4 *k16 = reinterpret_cast<uint4 *>(kt) + tid, *v16 = reinterpret_cast<uint4 *>(vt) + tid;
                if (rk != 1.f) *k16 = rescale_e4m3(*k16, rk);
                if (rv != 1.f) *v16 = rescale_e4m3(*v16, rv);
            }
        }
        if (mine) {
            const float ik = exp2i(1 - ek), iv = exp2i(1 - ev);
            uint8_t *kr = kt + (run.row + t) * kD, *vr = vt + (run.row + t) * kD;
            *reinterpret_cast<uint2 *>(kr + 8 * c) = pack_e4m3(y, ik);
            *reinterpret_cast<uint2 *>(kr + 64 + 8 * c) = pack_e4m3(y + 8, ik);
            const uint2 a = pack_e4m3(v, iv), b = pack_e4m3(v + 8, iv);
            *reinterpret_cast<uint4 *>(vr + 16 * c) = make_uint4(a.x, a.y, b.x, b.y);
        }
        if (tid == 0) {
            k_scale[tile] = exp2i(ek);
            v_scale[tile] = exp2i(ev);
        }
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
    // Measured with few / many (us, 10 heads; sequences x tokens): 1 x 4 4.7 / 5.9, 1 x 8 6.3 / 6.0, 1 x 64
    // 16.2 / 6.4, 1 x 2048 26.8 / 15.4, 16 x 4 6.1 / 6.8, 16 x 6 7.2 / 7.1, 16 x 8 8.0 / 7.1, 64 x 1 4.4 / 10.1,
    // 64 x 6 10.9 / 14.4, 64 x 8 11.8 / 14.3, 64 x 16 19.1 / 15.2: the border lies at 6 to 7 tokens a sequence
    // for few sequences, at some 11 for 64.
    if ((long long)n > 6ll * B) {
        // about two CTAs a SM: more would form the same sines more often
        const int groups = (int)min((long long)H + 1, max(1ll, 2ll * c.num_sms / (n / kBlock + B)));
        const int group = (H + 1 + groups - 1) / groups;
        rope_append_kv8_many_kernel<<<dim3((unsigned)runs, (unsigned)((H + 1 + group - 1) / group)), kManyThreads, 0,
                                      c.stream>>>(
            (const uint4 *)q, (const uint4 *)idx_q, (const uint4 *)k_new, (const uint4 *)v_new, (const uint4 *)idx_k_new,
            tok_pos, page_pos, start, bt, seq_lens, n, B, H, max_blocks, num_pages, group, (uint4 *)q_out,
            (uint4 *)idx_q_out, (uint8_t *)k_cache, (uint8_t *)v_cache, k_scale, v_scale, (uint4 *)idx_k_cache,
            rope_freqs(), dev_err);
        return cudaGetLastError();
    }
    rope_append_kv8_few_kernel<<<dim3((unsigned)runs, (unsigned)(H + 1)), kAppThreads, 0, c.stream>>>(
        (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)idx_q, (const __nv_bfloat16 *)k_new,
        (const __nv_bfloat16 *)v_new, (const __nv_bfloat16 *)idx_k_new, tok_pos, page_pos, start, bt, seq_lens, n, B, H,
        max_blocks, num_pages, (__nv_bfloat16 *)q_out, (__nv_bfloat16 *)idx_q_out, (uint8_t *)k_cache,
        (uint8_t *)v_cache, k_scale, v_scale, (__nv_bfloat16 *)idx_k_cache, rope_freqs(), dev_err);
    return cudaGetLastError();
}

}  // namespace uocr
