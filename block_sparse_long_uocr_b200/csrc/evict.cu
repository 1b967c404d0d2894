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
// Steps:
//   sums     total_j = sum_h mass[b][h][j] in fp64 (the order of two near totals does not depend on
//            the order of the heads' additions), as a key whose unsigned order is the totals'
//   select   the lowest kept key: the bin of 1/32 of an octave that holds it, then its rank
//            among that bin's keys (a bin of more than 512, such as that of the blocks that were
//            never attended: radix selection, 8 bits at a time from the highest bit in which the
//            keys differ); then, in block order, which columns stay and how many did before each
//   move     every kept column of totals and table to its new place
// In one launch, a cluster of CTAs per sequence: each holds a slice of the columns in shared memory
// and sends its keys to all; after one barrier each finds the threshold for itself (it is the same
// work, and no second barrier) and moves its slice.  All is read before any of it is written, so
// the outputs may be the inputs themselves; the totals are read and written once.  Tables too long
// for shared memory take three launches (sums; select; a CTA per row of totals that moves it in
// ascending pieces).
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
    const int w = lane < (int)(blockDim.x >> 5) ? s_w[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, w);
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + x - v;
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

// A candidate stays if key >> shift is above prefix, or is equal to it and among the first `need`
// such candidates; all: every equal one is.
struct Threshold {
    uint64_t prefix;
    int shift, need;
    bool all;
};
struct SelectSmem {
    int hist[kBins];
    uint64_t lo[32], hi[32];
    uint64_t prefix;
    int need, count;
};
// The threshold that keeps `take` of the candidates of [c0, c1) with use(key), fewer than there are,
// by a whole CTA.  load(j): the key of candidate j.
template <class Load, class Use>
__device__ __forceinline__ Threshold radix_threshold(SelectSmem &s, int c0, int c1, int take, Load load, Use use) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
    uint64_t lo = ~0ull, hi = 0;
    for (int j = c0 + tid; j < c1; j += n) {
        const uint64_t k = load(j);
        if (!use(k)) continue;
        lo = min(lo, k);
        hi = max(hi, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) {
        s.lo[warp] = lo;
        s.hi[warp] = hi;
    }
    __syncthreads();
    lo = lane < (n >> 5) ? s.lo[lane] : ~0ull;
    hi = lane < (n >> 5) ? s.hi[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    Threshold t;
    t.shift = 64 - __clzll(lo ^ hi);   // the bits above are the same in all keys
    t.prefix = t.shift < 64 ? hi >> t.shift : 0;
    t.need = take;
    t.all = false;
    while (t.shift > 0) {
        const int width = min(kDigit, t.shift), next = t.shift - width;
        for (int x = tid; x < kBins; x += n) s.hist[x] = 0;
        __syncthreads();
        for (int j0 = c0; j0 < c1; j0 += n) {   // whole warps take part
            const int j = j0 + tid;
            const uint64_t k = j < c1 ? load(j) : 0;
            const bool in = j < c1 && use(k) && (t.shift < 64 ? k >> t.shift : 0) == t.prefix;
            // lanes of one bin add together: most totals of a session are equal (0) or near
            const int bin = in ? (int)(k >> next) & ((1 << width) - 1) : -1;
            const unsigned same = __match_any_sync(0xffffffffu, bin);
            if (in && lane == __ffs(same) - 1) atomicAdd(&s.hist[bin], __popc(same));
        }
        __syncthreads();
        // the bin that holds the need-th highest, counted from the top bin
        if (tid < 32) {
            int c[kBins / 32], sum = 0;
#pragma unroll
            for (int x = 0; x < kBins / 32; ++x) sum += c[x] = s.hist[kBins - 1 - (tid * (kBins / 32) + x)];
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += y;
            }
            int before = incl - sum;
            if (before < t.need && t.need <= incl) {
#pragma unroll
                for (int x = 0; x < kBins / 32; ++x) {
                    if (before < t.need && t.need <= before + c[x]) {
                        s.prefix = t.prefix << width | (uint64_t)(kBins - 1 - (tid * (kBins / 32) + x));
                        s.need = t.need - before;
                        s.count = c[x];
                    }
                    before += c[x];
                }
            }
        }
        __syncthreads();
        t.prefix = s.prefix;
        t.need = s.need;
        t.shift = next;
        t.all = s.count == t.need;   // the whole bin stays: the bits below decide nothing
        if (t.all) break;
        __syncthreads();
    }
    return t;
}

// The lowest `n` set bits of `word`.
__device__ __forceinline__ unsigned lowest_bits(unsigned word, int n) {
    unsigned r = 0;
    for (; n > 0 && word; --n) {
        r |= word & (0u - word);
        word &= word - 1;
    }
    return r;
}

constexpr int kOneThreads = 1024;
constexpr int kOctBins = 4096;   // bins of 1/32 of an octave: 2^-64 .. 2^64
constexpr int kListMax = 512;
constexpr int kBinsEach = kOctBins / kOneThreads;

// The bin of a key, monotone in the key: everything below 2^-64 (negative totals and NaN too) falls
// in the first, everything from 2^64 on in the last.
__device__ __forceinline__ int octave_bin(uint64_t key) {
    if (!(key >> 63)) return 0;
    const int e32 = (int)((key & ~(1ull << 63)) >> 47);   // the exponent and 5 bits of the fraction
    return min(max(e32 - 32 * (1023 - 64), 0), kOctBins - 1);
}

// Sum over the CTA's threads; s_w holds a word per warp.
__device__ __forceinline__ int block_sum(int v, int *s_w) {
    v = __reduce_add_sync(0xffffffffu, v);
    const int lane = threadIdx.x & 31;
    if (lane == 0) s_w[threadIdx.x >> 5] = v;
    __syncthreads();
    const int sum = __reduce_add_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? s_w[lane] : 0);
    __syncthreads();   // s_w may be reused
    return sum;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

struct OneSmem {
    SelectSmem radix;
    int bins[kOctBins];
    uint64_t list[kListMax];
    int above[kListMax], same[kListMax];
    int w[32];
    int n_list, bin, bin_need, bin_count;
    Threshold t;
};

// The threshold from the keys, by a whole CTA of kOneThreads; s.bins zero at entry.
__device__ __forceinline__ Threshold octave_threshold(OneSmem &s, const uint64_t *keys, int c0, int c1, int take) {
    const int tid = threadIdx.x;
    for (int j0 = c0; j0 < c1; j0 += kOneThreads) {
        const int j = j0 + tid, bin = j < c1 ? octave_bin(keys[j]) : -1;
        // blocks that were never attended share the first bin
        const int zeros = __popc(__ballot_sync(0xffffffffu, bin == 0));
        if (bin > 0) atomicAdd(&s.bins[bin], 1);
        if ((tid & 31) == 0 && zeros) atomicAdd(&s.bins[0], zeros);
    }
    __syncthreads();
    // thread t counts its bins from the top down
    int c[kBinsEach], sum = 0, tot;
#pragma unroll
    for (int x = 0; x < kBinsEach; ++x) sum += c[x] = s.bins[kOctBins - 1 - kBinsEach * tid - x];
    if (tid == 0) s.n_list = 0;
    if (tid < kListMax) s.above[tid] = s.same[tid] = 0;
    int before = block_scan(sum, s.w, tot);
    if (before < take && take <= before + sum) {
#pragma unroll
        for (int x = 0; x < kBinsEach; ++x) {
            if (before < take && take <= before + c[x]) {
                s.bin = kOctBins - 1 - kBinsEach * tid - x;
                s.bin_need = take - before;
                s.bin_count = c[x];
            }
            before += c[x];
        }
    }
    __syncthreads();
    const int bin = s.bin, need = s.bin_need, count = s.bin_count;
    if (bin == 0) {   // mostly blocks of total 0: if they all are, they are ties
        bool other = false;
        for (int j = c0 + tid; j < c1; j += kOneThreads)
            other = other || (octave_bin(keys[j]) == 0 && keys[j] != order_key(0.0));
        if (!__syncthreads_or(other)) return Threshold{order_key(0.0), 0, need, need == count};
    }
    if (count > kListMax) {
        // (the keys above the bin are those with a higher bin: the same order)
        return radix_threshold(s.radix, c0, c1, need, [&](int j) { return keys[j]; },
                               [&](uint64_t k) { return octave_bin(k) == bin; });
    }
    for (int j = c0 + tid; j < c1; j += kOneThreads) {
        const uint64_t k = keys[j];
        if (octave_bin(k) == bin) s.list[atomicAdd(&s.n_list, 1)] = k;
    }
    __syncthreads();
    // every key's rank in the list: threads (key, part), the parts' counts added up
    const int parts = max(1, kOneThreads / max(count, 1));
    const int me = tid / parts;
    if (me < count) {
        const uint64_t k = s.list[me];
        int above = 0, same = 0;
#pragma unroll 4
        for (int x = tid - me * parts; x < count; x += parts) {
            const uint64_t o = s.list[x];
            above += o > k;
            same += o == k;
        }
        if (above) atomicAdd(&s.above[me], above);
        if (same) atomicAdd(&s.same[me], same);
    }
    __syncthreads();
    if (tid < count) {
        const int above = s.above[tid], same = s.same[tid];   // equal keys write the same
        if (above < need && need <= above + same) s.t = Threshold{s.list[tid], 0, need - above, need == above + same};
    }
    __syncthreads();
    return s.t;
}

constexpr int kMaxCluster = 8;

// Shared memory of the one-launch form: all keys, the slice's pages, kept columns and totals.
__host__ __device__ __forceinline__ int slice_columns(int max_blocks, int ctas) {
    return ((max_blocks + ctas - 1) / ctas + 31) / 32 * 32;
}
inline size_t one_smem(int H, int max_blocks, int ctas) {
    return (size_t)((max_blocks + 1) / 2 * 2) * 8 + (size_t)(H + 2) * slice_columns(max_blocks, ctas) * 4;
}

__global__ void __launch_bounds__(kOneThreads)
evict_one_kernel(const float *mass, const int32_t *table, const int32_t *seq_lens, int H, int max_blocks,
                 int keep_blocks, int n_sink, int ctas, int wide, int wide_out, float *new_mass, int32_t *new_table,
                 int32_t *new_lens, int32_t *__restrict__ freed, int32_t *__restrict__ n_freed, int32_t *dev_err) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ OneSmem s;
    const int rank = cluster_rank(), b = blockIdx.x / ctas, tid = threadIdx.x;
    const int slice = slice_columns(max_blocks, ctas);
    uint64_t *keys = reinterpret_cast<uint64_t *>(smem);
    int32_t *pages = reinterpret_cast<int32_t *>(keys + (max_blocks + 1) / 2 * 2);
    int *kept_cols = pages + slice;
    float *totals = reinterpret_cast<float *>(kept_cols + slice);   // [H][slice]
    for (int x = tid; x < kOctBins; x += kOneThreads) s.bins[x] = 0;
    cluster_arrive();
    const size_t row = (size_t)b * max_blocks;
    const int len = seq_lens[b], nb = causal_blocks(len, max_blocks);
    const int j0 = rank * slice, n = min(slice, max_blocks - j0);   // this CTA's columns (n may be <= 0)
    const float *src = mass + row * H + j0;
    float *dst = new_mass + row * H;

    if (nb <= keep_blocks) {   // nothing leaves (the same in every CTA of the cluster)
        cluster_wait();        // every CTA has read the length
        cluster_arrive();
        cluster_wait();
        if (nb < 0 && tid == 0 && rank == 0) flag_error(dev_err, UOCR_DEVERR_POS);
        for (int x = tid; x < n; x += kOneThreads) {
            new_table[row + j0 + x] = table[row + j0 + x];
            freed[row + j0 + x] = -1;
            if (mass != new_mass)
                for (int h = 0; h < H; ++h) dst[(size_t)h * max_blocks + j0 + x] = src[(size_t)h * max_blocks + x];
        }
        if (tid == 0 && rank == 0) {
            n_freed[b] = 0;
            new_lens[b] = len;
        }
        return;
    }

    // The slice into shared memory, every load in flight at once: 16 bytes each where the rows of the
    // arrays start on 16 bytes, else 4.
    if (wide) {
        for (int x = tid; x < (H + 1) * (slice / 4); x += kOneThreads) {
            const int h = x / (slice / 4), col = 4 * (x - h * (slice / 4));
            if (col >= n) continue;
            if (h < H)
                cp_async16(smem_addr(totals + h * slice + col), src + (size_t)h * max_blocks + col);
            else
                cp_async16(smem_addr(pages + col), table + row + j0 + col);
        }
    } else {
        for (int x = tid; x < n; x += kOneThreads) {
            for (int h = 0; h < H; ++h) cp_async4(smem_addr(totals + h * slice + x), src + (size_t)h * max_blocks + x);
            cp_async4(smem_addr(pages + x), table + row + j0 + x);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int gone = nb - keep_blocks;   // every such sequence is cut to keep_blocks
    const int all = ctas * kOneThreads, me = rank * kOneThreads + tid;
    for (int j = gone + me; j < max_blocks; j += all) freed[row + j] = -1;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // the totals' keys into every CTA's
    cluster_wait();   // every CTA has started
    const int c0 = n_sink, c1 = nb - kLocal;
    for (int x = max(0, c0 - j0) + tid; x < min(n, c1 - j0); x += kOneThreads) {
        double t = 0.0;
#pragma unroll 10
        for (int h = 0; h < H; ++h) t += (double)totals[h * slice + x];
        const uint64_t key = order_key(t);
        for (int y = 0; y < ctas; ++y) st_cluster(in_cta(keys + j0 + x, y), key);
    }
    cluster_arrive();
    cluster_wait();

    const int take = keep_blocks - kLocal - n_sink;   // of the candidates, fewer than there are
    Threshold t{~0ull, 0, 0, true};
    if (take > 0) t = octave_threshold(s, keys, c0, c1, take);
    const int edge = s.bin;
    // whether a column stays whatever the ties are, and whether it is one of them
    auto decide = [&](int j, bool &keep, bool &tie) {
        keep = j < max_blocks;
        tie = false;
        if (j < c0 || j >= c1) return;
        const uint64_t k = keys[j];
        const int bin = octave_bin(k);
        tie = take > 0 && bin == edge && k >> t.shift == t.prefix;
        keep = take > 0 && (bin > edge || (bin == edge && k >> t.shift > t.prefix) || (tie && t.all));
    };
    // kept columns and ties before the slice
    int kept = 0, ties = 0;
    for (int j = tid; j < min(j0, max_blocks); j += kOneThreads) {
        bool keep, tie;
        decide(j, keep, tie);
        kept += keep;
        ties += tie;
    }
    kept = block_sum(kept, s.w);
    if (!t.all) {
        ties = block_sum(ties, s.w);
        kept += min(ties, t.need);
    }
    // the slice's kept columns in order (two neighbours a thread and step); the others' pages go out
    const int kept0 = kept;
    for (int x0 = 0; x0 < n; x0 += 2 * kOneThreads) {
        const int x = x0 + 2 * tid;
        bool keep[2] = {false, false}, tie[2] = {false, false};
#pragma unroll
        for (int y = 0; y < 2; ++y)
            if (x + y < n) decide(j0 + x + y, keep[y], tie[y]);
        int tot;
        if (!t.all) {   // uniform over the cluster
            const int before = ties + block_scan(tie[0] + tie[1], s.w, tot);
            ties += tot;
            if (tie[0]) keep[0] = before < t.need;
            if (tie[1]) keep[1] = before + tie[0] < t.need;
        }
        int before = kept + block_scan(keep[0] + keep[1], s.w, tot);
        kept += tot;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            if (x + y >= n) break;
            if (keep[y])
                kept_cols[before++ - kept0] = x + y;
            else
                freed[row + (j0 + x + y - before)] = pages[x + y];
        }
    }
    __syncthreads();
    for (int i = tid; i < kept - kept0; i += kOneThreads) {
        const int x = kept_cols[i], to = kept0 + i;
        new_table[row + to] = pages[x];
#pragma unroll 10
        for (int h = 0; h < H; ++h) dst[(size_t)h * max_blocks + to] = totals[h * slice + x];
    }
    // behind the kept columns (4 at a time where the outputs' rows start on 16 bytes)
    const int end = max_blocks - gone;
    if (wide_out) {
        const int quads = (max_blocks - end) / 4;   // the quads from the row's end down to `end`
        for (int x = me; x < (H + 1) * quads; x += all) {
            const int h = x / quads, j = max_blocks - 4 * (x - h * quads + 1);
            if (h < H)
                *reinterpret_cast<float4 *>(dst + (size_t)h * max_blocks + j) = make_float4(0.f, 0.f, 0.f, 0.f);
            else
                *reinterpret_cast<int4 *>(new_table + row + j) = make_int4(-1, -1, -1, -1);
        }
    }
    const int rest = wide_out ? (max_blocks - end) % 4 : max_blocks - end;
    for (int j = end + me; j < end + rest; j += all) {
        new_table[row + j] = -1;
        for (int h = 0; h < H; ++h) dst[(size_t)h * max_blocks + j] = 0.f;
    }
    if (me == 0) {
        n_freed[b] = gone;
        new_lens[b] = len - gone * kBlock;
    }
}

// dst[j]: the new place of column j, or -1 for a removed one.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const uint64_t *__restrict__ keys, const int32_t *table, const int32_t *seq_lens, int max_blocks,
                    int keep_blocks, int n_sink, int32_t *__restrict__ dst, int32_t *new_table, int32_t *new_lens,
                    int32_t *__restrict__ freed, int32_t *__restrict__ n_freed, int32_t *dev_err) {
    __shared__ SelectSmem s_sel;
    __shared__ int s_w[32];
    const int b = blockIdx.x, tid = threadIdx.x;
    const size_t row = (size_t)b * max_blocks;
    pdl_wait();
    const int len = seq_lens[b];
    const int nb = causal_blocks(len, max_blocks);
    if (nb < 0 && tid == 0) flag_error(dev_err, UOCR_DEVERR_POS);
    const bool cut_any = nb > keep_blocks;
    const int c0 = n_sink, c1 = nb - kLocal;          // candidates [c0, c1)
    const int take = keep_blocks - kLocal - n_sink;   // kept of them: fewer than there are
    Threshold t{~0ull, 0, 0, true};
    if (cut_any && take > 0)
        t = radix_threshold(s_sel, c0, c1, take, [&](int j) { return __ldcg(keys + row + j); },
                            [](uint64_t) { return true; });

    int kept = 0, ties = 0, gone = 0;   // before the piece
    for (int j0 = 0; j0 < max_blocks; j0 += kSelThreads) {
        const int j = j0 + tid;
        const bool in = j < max_blocks;
        const int page = in ? table[row + j] : -1;
        bool keep = in, tie = false;
        if (cut_any && j >= c0 && j < c1) {
            const uint64_t k = take > 0 ? __ldcg(keys + row + j) >> t.shift : 0;
            tie = take > 0 && k == t.prefix;
            keep = take > 0 && k > t.prefix;
        }
        int tot_tie = 0, tot_keep;
        if (cut_any) {   // uniform over the CTA
            const int before = block_scan(tie ? 1 : 0, s_w, tot_tie);
            if (tie) keep = ties + before < t.need;
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

namespace {
// CTAs per sequence of the one-launch form (a CTA takes an SM's threads): at most 4, as long as all
// sequences' fit on the SMs at once, and more where only a smaller slice fits in shared memory; 0
// where none does.  Measured with 1 / 2 / 4 / 8 CTAs and with three launches (us; sequences x blocks, 10
// heads unless given): 1 x 4096 - / 12.4 / 10.9 / 10.2, 20.7; 8 x 4096 - / 12.7 / 11.1 / 10.5, 21.6; 64 x 4096
// - / 13.2 / 21.8 / 40.4, 26.9; 32 x 2048 10.9 / 9.5 / 9.0 / 18.6, 17.5; 16 x 2048 (16 heads) 13.3 / 11.1 / 9.9 /
// 13.8, 16.7; 64 x 1024 8.7 / 7.9 / 14.7 / 30.9, 17.5; 128 x 512 7.7 / 13.9 / 26.5 / 52.9, 18.9; 3 x 777 (12
// heads) 8.2 / 7.8 / 7.8 / 7.8, 11.1.  Three launches where nothing fits: 8 x 20480 68, 16 x 32768 131 (floors
// 2.3 and 7.4: one CTA a sequence selects, one a row moves).
constexpr size_t kRoom = 192 * 1024;   // shared memory of the slice and the keys
int evict_ctas(int B, int H, int max_blocks, int num_sms) {
    int ctas = 4;
    while (ctas > 1 && (long long)B * ctas > num_sms && one_smem(H, max_blocks, ctas / 2) <= kRoom) ctas /= 2;
    while (ctas < kMaxCluster && one_smem(H, max_blocks, ctas) > kRoom) ctas *= 2;
    return one_smem(H, max_blocks, ctas) <= kRoom ? ctas : 0;
}
}  // namespace

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
    cudaLaunchConfig_t cfg = {};
    cfg.stream = c.stream;
    const int ctas = evict_ctas(B, H, max_blocks, c.num_sms);
    if (ctas > 0) {
        const size_t smem = one_smem(H, max_blocks, ctas);
        // the same for every call: another thread's call for a smaller table must not lower it before this launch
        cudaError_t e = cudaFuncSetAttribute(evict_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRoom);
        if (e != cudaSuccess) return e;
        const int wide = max_blocks % 4 == 0 && ((uintptr_t)mass | (uintptr_t)table) % 16 == 0;
        const int wide_out = max_blocks % 4 == 0 && ((uintptr_t)new_mass | (uintptr_t)new_table) % 16 == 0;
        cudaLaunchAttribute cl[1];
        cl[0].id = cudaLaunchAttributeClusterDimension;
        cl[0].val.clusterDim.x = ctas;
        cl[0].val.clusterDim.y = cl[0].val.clusterDim.z = 1;
        cfg.attrs = cl;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)(B * ctas));
        cfg.blockDim = dim3(kOneThreads);
        cfg.dynamicSmemBytes = smem;
        return cudaLaunchKernelEx(&cfg, evict_one_kernel, mass, table, seq_lens, H, max_blocks, keep_blocks, n_sink,
                                  ctas, wide, wide_out, new_mass, new_table, new_lens, freed, n_freed, dev_err);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
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
