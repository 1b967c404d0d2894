// kv8_attn.cu -- decode attention over a key / value cache held in e4m3, with a scale for each
// (page, head): over the 16 selected blocks of a query, or over a prefix and the local window.
//
// The same steps as the bf16 forms (sparse_attn.cu, dense_attn.cu; Unlimited-OCR-2 walk-through,
// news.rkmt.cn/news/25027, section 五 step 4) on half the bytes:
//   z_t = scale * ks * (q . k8_t),  w = softmax(z) over the visible tokens,  out = sum_t w_t vs v8_t
// with ks, vs the scales of the token's (page, head).  Optionally each block's share of the
// softmax, sum_{t in block} w_t, is added to a running total per (sequence, head, block): what
// block eviction ranks by.  A total has one writer per call, so its order of additions is fixed.
#include <math.h>

#include "kernels.h"
#include "kv8.cuh"

namespace uocr {

namespace {

// A warp's softmax state over one or more blocks: acc of lane (g, 0) holds dims 16 g .. 16 g + 15.
struct State8 {
    float m = -INFINITY, l = 0.f;
    float acc[16];
    __device__ __forceinline__ State8() {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    }
};

// One block: scores, softmax weights against the running maximum, weighted values.  Returns the
// block's weight sum in units of 2^m (the state's new maximum).  `visible` >= 1 tokens count.
__device__ __forceinline__ float attend8(State8 &st, const uint4 (&k)[8], uint4 (&v)[8], const Query8 &q, float ks,
                                         float vs, float scale_log2, int visible, int lane) {
    float z[4];
    scores8(z, k, q, lane);
    const float f = ks * scale_log2;
    const int g = lane >> 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = z[i] * q.unit * f;
    if (visible < kBlock) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * i + g >= visible) z[i] = -INFINITY;
        mask_v8(v, visible, lane);
    }
    float mb = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, x));
    const float m = fmaxf(st.m, mb);
    const float base = m == -INFINITY ? 0.f : m;      // every score -inf: weights 0, not NaN
    const float corr = exp2f(st.m - base);            // 0 on the first block
    float p[4], lb = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = exp2f(z[i] - base);
        lb += p[i];
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) lb += __shfl_xor_sync(0xffffffffu, lb, x);
    st.m = m;
    st.l = fmaf(st.l, corr, lb);
#pragma unroll
    for (int e = 0; e < 16; ++e) st.acc[e] *= corr;
    weighted_sum8(st.acc, p, v, vs, lane);
    return lb;
}

// Warp states merged over a CTA's warps.  s_acc [warps][128], s_ml [warps] {m, l}.
template <int kWarps>
struct Merge8 {
    float acc[kWarps][kD];
    float2 ml[kWarps];
};
template <int kWarps>
__device__ __forceinline__ void put_state8(Merge8<kWarps> &s, const State8 &st, int warp, int lane) {
    if (lane == 0) s.ml[warp] = make_float2(st.m, st.l);
    if ((lane & 3) == 0) {
        float4 *dst = reinterpret_cast<float4 *>(&s.acc[warp][16 * (lane >> 2)]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            dst[e] = make_float4(st.acc[4 * e], st.acc[4 * e + 1], st.acc[4 * e + 2], st.acc[4 * e + 3]);
    }
}

__device__ __forceinline__ int checked_page(const int32_t *bt_row, int j, int num_pages, int lane, int32_t *dev_err) {
    const int page = __ldg(bt_row + j);
    if ((unsigned)page < (unsigned)num_pages) return page;
    if (lane == 0) flag_error(dev_err, UOCR_DEVERR_PAGE);
    return -1;
}

constexpr int kSWarps = kSel;   // sparse: a warp per selected block
constexpr int kDWarps = 4;      // dense: warps of a CTA, each every fourth block of its chunk
constexpr int kDChunk = 16;     // dense: blocks of a chunk

}  // namespace

// A CTA per (query, head), a warp per selection slot.
__global__ void __launch_bounds__(kSWarps * 32)
sparse_attn_kv8_kernel(const uint4 *__restrict__ q, const uint4 *__restrict__ kc, const uint4 *__restrict__ vc,
                       const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                       const int32_t *__restrict__ bt, const int32_t *__restrict__ seq_lens,
                       const int32_t *__restrict__ q_seq, const int32_t *__restrict__ q_pos,
                       const int32_t *__restrict__ sel, int B, int H, int max_blocks, int num_pages,
                       float scale_log2, int implicit_local, __nv_bfloat16 *__restrict__ out,
                       float *__restrict__ mass, int32_t *dev_err) {
    __shared__ __align__(16) Merge8<kSWarps> s;
    __shared__ int s_j[kSWarps];
    const int ih = blockIdx.x, i = ih / H, h = ih - i * H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    QueryRef r;
    const bool ok = resolve_query(i, seq_lens, q_seq, q_pos, B, max_blocks, dev_err, threadIdx.x == 0 && h == 0, r);
    int j = -2;
    if (ok && implicit_local) {   // slots that do not depend on the scores (see sparse_attn.cu)
        if (r.nb <= kSel)
            j = warp < r.nb ? warp : -1;
        else if (warp >= kRemote)
            j = r.nb - kSel + warp;
    }
    if (j == -2) {
        pdl_wait();
        j = ok ? __ldg(sel + (size_t)i * kSel + warp) : -1;
    }
    if (j >= 0 && j >= r.nb) {
        if (lane == 0) flag_error(dev_err, UOCR_DEVERR_SEL);
        j = -1;
    }
    const int page = j >= 0 ? checked_page(bt + (size_t)r.b * max_blocks, j, num_pages, lane, dev_err) : -1;

    State8 st;
    if (page >= 0) {
        const size_t tile = (size_t)page * H + h;
        uint4 k[8], v[8];
        load_k8(k, kc + tile * kTile8U4, lane);
        load_v8(v, vc + tile * kTile8U4, lane);
        const float ks = __ldg(k_scale + tile), vs = __ldg(v_scale + tile);
        const Query8 qf = load_query8(q + (size_t)ih * (kD / 8), lane);
        attend8(st, k, v, qf, ks, vs, scale_log2, min(kBlock, r.p - j * kBlock + 1), lane);
    }
    put_state8(s, st, warp, lane);
    if (lane == 0) s_j[warp] = page >= 0 ? j : -1;
    __syncthreads();

    if (threadIdx.x < kD) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kSWarps; ++w) M = fmaxf(M, s.ml[w].x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f, A = 0.f;
#pragma unroll
        for (int w = 0; w < kSWarps; ++w) {
            const float f = exp2f(s.ml[w].x - base);   // 0 for an empty slot
            L = fmaf(s.ml[w].y, f, L);
            A = fmaf(s.acc[w][threadIdx.x], f, A);
        }
        // L is 0 for a query without a visible token, NaN where a score is
        out[(size_t)ih * kD + threadIdx.x] = __float2bfloat16_rn(L != 0.f ? A / L : 0.f);
        if (mass && threadIdx.x < kSWarps && s_j[threadIdx.x] >= 0) {
            // one writer per block: the first slot that names it adds the weights of all that do
            const int mine = s_j[threadIdx.x];
            bool first = true;
            float w = 0.f;
#pragma unroll
            for (int x = 0; x < kSWarps; ++x) {
                if (s_j[x] != mine) continue;
                if (x < (int)threadIdx.x) first = false;
                w += s.ml[x].y * exp2f(s.ml[x].x - base);
            }
            if (first && L > 0.f) {
                float *m = mass + ((size_t)r.b * H + h) * max_blocks + mine;
                *m += finite_weight(w / L);
            }
        }
    }
    // warps whose blocks were known in advance did not wait for the selection kernel: this grid
    // still completes after it
    if (blockIdx.x == 0 && threadIdx.x == 0) pdl_wait();
}

// Split over chunks of 16 blocks: CTA (query, head, chunk) leaves {m, l}, acc[128] and, for the
// totals, each block's weight sum with the maximum it refers to.
__global__ void __launch_bounds__(kDWarps * 32)
dense_kv8_chunk_kernel(const uint4 *__restrict__ q, const uint4 *__restrict__ kc, const uint4 *__restrict__ vc,
                       const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                       const int32_t *__restrict__ bt, const int32_t *__restrict__ seq_lens, int B, int H,
                       int max_blocks, int num_pages, int ref_blocks, int n_chunks, float scale_log2,
                       float *__restrict__ part_acc, float2 *__restrict__ part_ml, float2 *__restrict__ blk_ml,
                       int32_t *dev_err) {
    __shared__ __align__(16) Merge8<kDWarps> s;
    const int chunk = blockIdx.x % n_chunks, ih = blockIdx.x / n_chunks;
    const int i = ih / H, h = ih - i * H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    QueryRef r;
    const bool ok = resolve_query(i, seq_lens, nullptr, nullptr, B, max_blocks, dev_err,
                                  threadIdx.x == 0 && chunk == 0 && h == 0, r);
    const int nb = ok ? r.nb : 0;
    if (chunk * kDChunk >= nb) return;   // the merge reads only the chunks below nb

    const Query8 qf = load_query8(q + (size_t)ih * (kD / 8), lane);
    const int32_t *bt_row = bt + (size_t)r.b * max_blocks;
    State8 st;
    for (int x = warp; x < kDChunk; x += kDWarps) {
        const int j = chunk * kDChunk + x;
        if (j >= nb) break;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (j < ref_blocks || j >= nb - kLocal) {
            const int page = checked_page(bt_row, j, num_pages, lane, dev_err);
            if (page >= 0) {
                const size_t tile = (size_t)page * H + h;
                uint4 k[8], v[8];
                load_k8(k, kc + tile * kTile8U4, lane);
                load_v8(v, vc + tile * kTile8U4, lane);
                const float ks = __ldg(k_scale + tile), vs = __ldg(v_scale + tile);
                ml.y = attend8(st, k, v, qf, ks, vs, scale_log2, min(kBlock, r.p - j * kBlock + 1), lane);
                ml.x = st.m;
            }
        }
        if (blk_ml && lane == 0) blk_ml[(size_t)ih * max_blocks + j] = ml;
    }
    put_state8(s, st, warp, lane);
    __syncthreads();
    const int d = threadIdx.x;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDWarps; ++w) M = fmaxf(M, s.ml[w].x);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, A = 0.f;
#pragma unroll
    for (int w = 0; w < kDWarps; ++w) {
        const float f = exp2f(s.ml[w].x - base);
        L = fmaf(s.ml[w].y, f, L);
        A = fmaf(s.acc[w][d], f, A);
    }
    const size_t slot = (size_t)ih * n_chunks + chunk;
    part_acc[slot * kD + d] = A;
    if (d == 0) part_ml[slot] = make_float2(M, L);
}

// CTA (query, head, 0) merges the chunks' states into the output; CTA (query, head, 1 + x) adds the
// weights of the blocks [128 x, 128 x + 128) to their totals.
__global__ void __launch_bounds__(kD)
dense_kv8_merge_kernel(const int32_t *__restrict__ seq_lens, int B, int H, int max_blocks, int n_chunks, int parts,
                       const float *__restrict__ part_acc, const float2 *__restrict__ part_ml,
                       const float2 *__restrict__ blk_ml, __nv_bfloat16 *__restrict__ out, float *__restrict__ mass) {
    __shared__ float s_red[kD / 32];
    const int ih = blockIdx.x / parts, part = blockIdx.x - ih * parts;
    const int i = ih / H, d = threadIdx.x;
    QueryRef r;
    const bool ok = resolve_query(i, seq_lens, nullptr, nullptr, B, max_blocks, nullptr, false, r);
    const int nb = ok ? r.nb : 0;
    const int used = (nb + kDChunk - 1) / kDChunk;
    pdl_wait();
    if (part > 0 && (part - 1) * kD >= nb) return;
    const float2 *ml = part_ml + (size_t)ih * n_chunks;
    float M = -INFINITY;
    for (int c = d; c < used; c += kD) M = fmaxf(M, ml[c].x);
    M = warp_max(M);
    if ((d & 31) == 0) s_red[d >> 5] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    __syncthreads();
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int c = d; c < used; c += kD) L += ml[c].y * exp2f(ml[c].x - base);
    L = warp_sum(L);
    if ((d & 31) == 0) s_red[d >> 5] = L;
    __syncthreads();
    L = s_red[0] + s_red[1] + s_red[2] + s_red[3];
    if (part == 0) {
        float A = 0.f;
#pragma unroll 8
        for (int c = 0; c < used; ++c)
            A = fmaf(part_acc[((size_t)ih * n_chunks + c) * kD + d], exp2f(ml[c].x - base), A);
        out[(size_t)ih * kD + d] = __float2bfloat16_rn(L != 0.f ? A / L : 0.f);
    } else if (L > 0.f) {
        const int j = (part - 1) * kD + d;
        if (j < nb) {
            const float2 b = blk_ml[(size_t)ih * max_blocks + j];
            mass[(size_t)ih * max_blocks + j] += finite_weight(b.y * exp2f(b.x - base) / L);
        }
    }
}

// ------------------------------------------------------------------ host side
cudaError_t launch_sparse_attn_kv8(const LaunchCtx &c, const void *q, const Kv8Cache &kv, const int32_t *bt,
                                   const int32_t *seq_lens, const int32_t *q_seq, const int32_t *q_pos,
                                   const int32_t *sel, int n_q, int B, int H, int max_blocks, int num_pages,
                                   float scale, void *out, float *mass, bool implicit_local, int32_t *dev_err) {
    const long long grid = (long long)n_q * H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kSWarps * 32);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = c.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, sparse_attn_kv8_kernel, (const uint4 *)q, (const uint4 *)kv.k, (const uint4 *)kv.v,
                              kv.k_scale, kv.v_scale, bt, seq_lens, q_seq, q_pos, sel, B, H, max_blocks, num_pages,
                              scale * kLog2e, implicit_local ? 1 : 0, (__nv_bfloat16 *)out, mass, dev_err);
}

namespace {
struct Dense8Ws {
    size_t acc_off, ml_off, blk_off, total;
};
Dense8Ws dense8_layout(int n_q, int H, int max_blocks) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)n_q * H, slots = rows * ((max_blocks + kDChunk - 1) / kDChunk);
    Dense8Ws w{};
    w.ml_off = up(slots * kD * 4);
    w.blk_off = w.ml_off + up(slots * sizeof(float2));
    w.total = w.blk_off + up(rows * max_blocks * sizeof(float2));
    return w;
}
}  // namespace

size_t dense_kv8_workspace(int n_q, int H, int max_blocks) { return dense8_layout(n_q, H, max_blocks).total; }

cudaError_t launch_dense_kv8(const LaunchCtx &c, const void *q, const Kv8Cache &kv, const int32_t *bt,
                             const int32_t *seq_lens, int B, int H, int max_blocks, int num_pages, int ref_blocks,
                             float scale, void *out, float *mass, void *ws, int32_t *dev_err) {
    const Dense8Ws w = dense8_layout(B, H, max_blocks);
    const int n_chunks = (max_blocks + kDChunk - 1) / kDChunk;
    float *acc = (float *)((char *)ws + w.acc_off);
    float2 *ml = (float2 *)((char *)ws + w.ml_off);
    float2 *blk = mass ? (float2 *)((char *)ws + w.blk_off) : nullptr;
    const long long grid = (long long)B * H * n_chunks;
    const int parts = mass ? 1 + (max_blocks + kD - 1) / kD : 1;
    if (grid > 0x7fffffffLL || (long long)B * H * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kDWarps * 32);
    cfg.stream = c.stream;
    cudaError_t e = cudaLaunchKernelEx(&cfg, dense_kv8_chunk_kernel, (const uint4 *)q, (const uint4 *)kv.k,
                                       (const uint4 *)kv.v, kv.k_scale, kv.v_scale, bt, seq_lens, B, H, max_blocks,
                                       num_pages, ref_blocks, n_chunks, scale * kLog2e, acc, ml, blk, dev_err);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(B * H * parts));
    cfg.blockDim = dim3(kD);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dense_kv8_merge_kernel, seq_lens, B, H, max_blocks, n_chunks, parts,
                              (const float *)acc, (const float2 *)ml, (const float2 *)blk, (__nv_bfloat16 *)out, mass);
}

}  // namespace uocr
