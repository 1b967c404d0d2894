// evict.cu -- eviction of KV blocks by accumulated attention weight.
//
// The decode and prefill attention over the 8-bit cache add each block's softmax weight to a
// running total mass[b][h][j].  When a sequence has more than keep_blocks causal blocks, this
// keeps its first n_sink blocks, its 4 local ones (the window that every query attends) and, of
// the others, those with the highest total over the heads, the lower block id on ties (the order
// of the block selection); the others' columns are taken out of the block table and the totals,
// everything behind a removed column moves down, and the sequence gets shorter by 32 tokens per
// removed block.  Cached keys carry their rotation, and rope_append takes positions as arguments,
// so blocks may move in the table without touching the cache.
//
// Steps, one kernel each:
//   sums     total_j = sum_h mass[b][h][j] in fp64 (the order of two near totals does not depend on
//            the order of the heads' additions), as a key whose unsigned order is the totals'
//   select   a CTA per sequence: radix selection of the lowest kept key, then one pass in block
//            order that gives every column its new place, the freed pages, the table and the length
//   compact  a CTA per (sequence, head) moves a row of totals in ascending pieces, each read before
//            it is written, so that the outputs may be the inputs themselves
// Bytes: the totals are read twice and written once.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace uocr {

namespace {
constexpr int kSumThreads = 128;
constexpr int kSelThreads = 1024;
constexpr int kDigit = 8;
constexpr int kBins = 1 << kDigit;
constexpr int kCompThreads = 512;

// Unsigned order of fp64: greater total, greater key; NaN below everything, -0 as +0.
__device__ __forceinline__ uint64_t order_key(double t) {
    if (t != t) return 0;
    const long long b = __double_as_longlong(t + 0.0);
    return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

// A sequence's causal blocks, or -1 for a length that the table cannot hold.
__device__ __forceinline__ int causal_blocks(int len, int max_blocks) {
    return len < 0 || len > max_blocks * kBlock ? -1 : (len + kBlock - 1) / kBlock;
}

// Exclusive prefix sum over the CTA's threads and the total; s_w holds a word per warp.
__device__ __forceinline__ int block_scan(int v, int *s_w, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int n = blockDim.x >> 5;
        int w = lane < n ? s_w[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        if (lane < n) s_w[lane] = w;
    }
    __syncthreads();
    const int before = (warp ? s_w[warp - 1] : 0) + x - v;
    total = s_w[(blockDim.x >> 5) - 1];
    __syncthreads();   // s_w may be reused
    return before;
}
}  // namespace

__global__ void __launch_bounds__(kSumThreads)
evict_sum_kernel(const float *__restrict__ mass, const int32_t *__restrict__ seq_lens, int H, int max_blocks,
                 int chunks, int keep_blocks, uint64_t *__restrict__ keys) {
    const int b = blockIdx.x / chunks;
    const int j = (blockIdx.x - b * chunks) * kSumThreads + threadIdx.x;
    const int nb = causal_blocks(__ldg(seq_lens + b), max_blocks);
    if (nb <= keep_blocks || j >= nb) return;
    const float *src = mass + (size_t)b * H * max_blocks + j;
    double t = 0.0;
#pragma unroll 8
    for (int h = 0; h < H; ++h) t += (double)__ldg(src + (size_t)h * max_blocks);
    keys[(size_t)b * max_blocks + j] = order_key(t);
}

// dst[j]: the new place of column j, or -1 for a removed one.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const uint64_t *__restrict__ keys, const int32_t *table, const int32_t *seq_lens, int max_blocks,
                    int keep_blocks, int n_sink, int32_t *__restrict__ dst, int32_t *new_table, int32_t *new_lens,
                    int32_t *__restrict__ freed, int32_t *__restrict__ n_freed, int32_t *dev_err) {
    __shared__ int s_hist[kBins];
    __shared__ int s_w[32];
    __shared__ uint64_t s_prefix;
    __shared__ int s_need;
    const int b = blockIdx.x, tid = threadIdx.x;
    const size_t row = (size_t)b * max_blocks;
    pdl_wait();
    const int len = seq_lens[b];
    const int nb = causal_blocks(len, max_blocks);
    if (nb < 0 && tid == 0) flag_error(dev_err, UOCR_DEVERR_POS);
    const bool cut_any = nb > keep_blocks;
    const int c0 = n_sink, c1 = nb - kLocal;          // candidates [c0, c1)
    const int take = keep_blocks - kLocal - n_sink;   // kept of them: fewer than there are

    // the take-th highest key T, and how many candidates equal to T are kept
    uint64_t prefix = 0;
    int need = cut_any ? take : 0;
    if (cut_any && take > 0) {
        for (int shift = 64 - kDigit; shift >= 0; shift -= kDigit) {
            if (tid < kBins) s_hist[tid] = 0;
            __syncthreads();
            const uint64_t mask = shift == 64 - kDigit ? 0 : ~0ull << (shift + kDigit);
            for (int j = c0 + tid; j < c1; j += kSelThreads) {
                const uint64_t k = __ldcg(keys + row + j);
                if ((k & mask) == prefix) atomicAdd(&s_hist[(int)(k >> shift) & (kBins - 1)], 1);
            }
            __syncthreads();
            // the bin that holds the need-th highest, counted from the top bin
            if (tid < 32) {
                int c[kBins / 32], sum = 0;
#pragma unroll
                for (int x = 0; x < kBins / 32; ++x) sum += c[x] = s_hist[kBins - 1 - (tid * (kBins / 32) + x)];
                int incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (tid >= o) incl += y;
                }
                int before = incl - sum;
                if (before < need && need <= incl) {
#pragma unroll
                    for (int x = 0; x < kBins / 32; ++x) {
                        if (need <= before + c[x]) {
                            s_prefix = prefix | (uint64_t)(kBins - 1 - (tid * (kBins / 32) + x)) << shift;
                            s_need = need - before;
                            break;
                        }
                        before += c[x];
                    }
                }
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
    }

    int kept = 0, ties = 0, gone = 0;   // before the piece
    for (int j0 = 0; j0 < max_blocks; j0 += kSelThreads) {
        const int j = j0 + tid;
        const bool in = j < max_blocks;
        const int page = in ? table[row + j] : -1;
        bool keep = in, tie = false;
        if (cut_any && j >= c0 && j < c1) {
            const uint64_t k = take > 0 ? __ldcg(keys + row + j) : 0;
            tie = take > 0 && k == prefix;
            keep = take > 0 && k > prefix;
        }
        int tot_tie = 0, tot_keep;
        if (cut_any) {   // uniform over the CTA
            const int t = block_scan(tie ? 1 : 0, s_w, tot_tie);
            if (tie) keep = ties + t < need;
        }
        const int at = block_scan(keep ? 1 : 0, s_w, tot_keep);   // also: the piece is read before it is written
        if (in) {
            dst[row + j] = keep ? kept + at : -1;
            if (keep)
                new_table[row + kept + at] = page;
            else
                freed[row + gone + tid - at] = page;
        }
        ties += tot_tie;
        kept += tot_keep;
        gone += min(kSelThreads, max_blocks - j0) - tot_keep;
    }
    __syncthreads();
    for (int j = kept + tid; j < max_blocks; j += kSelThreads) new_table[row + j] = -1;
    for (int j = gone + tid; j < max_blocks; j += kSelThreads) freed[row + j] = -1;
    if (tid == 0) {
        n_freed[b] = gone;
        new_lens[b] = len - gone * kBlock;
    }
}

__global__ void __launch_bounds__(kCompThreads)
evict_compact_kernel(const float *mass, const int32_t *__restrict__ dst, const int32_t *__restrict__ n_freed, int H,
                     int max_blocks, float *new_mass) {
    const int bh = blockIdx.x, b = bh / H;
    const float *src = mass + (size_t)bh * max_blocks;
    float *out = new_mass + (size_t)bh * max_blocks;
    const int32_t *d = dst + (size_t)b * max_blocks;
    pdl_wait();
    const int gone = __ldcg(n_freed + b);
    if (gone == 0 && mass == new_mass) return;
    constexpr int kPer = 4;
    for (int j0 = 0; j0 < max_blocks; j0 += kCompThreads * kPer) {
        float v[kPer];
        int to[kPer];
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int j = j0 + x * kCompThreads + threadIdx.x;
            to[x] = j < max_blocks ? __ldcg(d + j) : -1;
            v[x] = to[x] >= 0 ? src[j] : 0.f;
        }
        __syncthreads();   // places move down: the piece is read before any of it is written
#pragma unroll
        for (int x = 0; x < kPer; ++x)
            if (to[x] >= 0) out[to[x]] = v[x];
        __syncthreads();
    }
    for (int j = max_blocks - gone + threadIdx.x; j < max_blocks; j += kCompThreads) out[j] = 0.f;
}

size_t evict_workspace(int B, int max_blocks) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    return up((size_t)B * max_blocks * 8) + up((size_t)B * max_blocks * 4);
}

cudaError_t launch_evict(const LaunchCtx &c, const float *mass, const int32_t *table, const int32_t *seq_lens, int B,
                         int H, int max_blocks, int keep_blocks, int n_sink, float *new_mass, int32_t *new_table,
                         int32_t *new_lens, int32_t *freed, int32_t *n_freed, void *ws, int32_t *dev_err) {
    uint64_t *keys = (uint64_t *)ws;
    int32_t *dst = (int32_t *)((char *)ws + ((size_t)B * max_blocks * 8 + 255) / 256 * 256);
    const int chunks = (max_blocks + kSumThreads - 1) / kSumThreads;
    if ((long long)B * chunks > 0x7fffffffLL || (long long)B * H > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = c.stream;
    cfg.gridDim = dim3((unsigned)(B * chunks));
    cfg.blockDim = dim3(kSumThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_sum_kernel, mass, seq_lens, H, max_blocks, chunks, keep_blocks, keys);
    if (e != cudaSuccess) return e;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)B);
    cfg.blockDim = dim3(kSelThreads);
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, (const uint64_t *)keys, table, seq_lens, max_blocks, keep_blocks,
                           n_sink, dst, new_table, new_lens, freed, n_freed, dev_err);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(B * H));
    cfg.blockDim = dim3(kCompThreads);
    return cudaLaunchKernelEx(&cfg, evict_compact_kernel, mass, (const int32_t *)dst, (const int32_t *)n_freed, H,
                              max_blocks, new_mass);
}

}  // namespace uocr
