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

constexpr float kLeast = -3.4028235e38f;   // the maximum over nothing: finite, so that it can be subtracted

// A warp's softmax state over one or more blocks: acc of lane (g, 0) holds dims 16 g .. 16 g + 15.
struct State8 {
    float m = kLeast, l = 0.f;
    float acc[16];
    __device__ __forceinline__ State8() {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    }
};

// The blocks that a warp attends: lane t holds the t-th block's id, its page (-1: none) and scales.
struct Blocks8 {
    int j, page;
    float ks, vs;
};

// The scales of the lane's block; by a whole warp, after j and page are set.  They are not used
// before the first block's K and V are on their way: a product with them here would wait for them
// first (0.5 us of a call that takes 4.5).
__device__ __forceinline__ void load_scales8(Blocks8 &bl, const float *__restrict__ k_scale,
                                             const float *__restrict__ v_scale, int H, int h) {
    const size_t tile = (size_t)max(bl.page, 0) * H + h;
    bl.ks = bl.page >= 0 ? __ldg(k_scale + tile) : 0.f;
    bl.vs = bl.page >= 0 ? __ldg(v_scale + tile) : 0.f;
}

// Attention over the warp's blocks with a running maximum; done(t, m, l): the t-th block's weight
// sum l in units of 2^m.  A block's weights are taken against its own maximum and meet the others' as
// fp32 factors: against the running one, fp16 would keep few bits of the weights of a block far below
// it, which count where its value scale is far above the others'.
// A block's K and V are loaded together and used at once; what overlaps the arithmetic are the other
// warps' loads (16 to 20 a SM).  Loading the next block's K into the registers that the scores free was
// slower (266 against 215 us for 16 x 32768 tokens): it keeps 32 more registers alive through the
// weighted sum, which then spills.
template <class Done>
__device__ __forceinline__ void attend8(State8 &st, const Blocks8 &bl, const uint4 *__restrict__ kc,
                                        const uint4 *__restrict__ vc, int H, int h, int p, float scale_log2,
                                        const Query8 &q, int lane, Done done) {
    const int g = lane >> 2;
    for (unsigned left = __ballot_sync(0xffffffffu, bl.page >= 0); left; left &= left - 1) {
        const int t = __ffs(left) - 1;
        const size_t at = ((size_t)__shfl_sync(0xffffffffu, bl.page, t) * H + h) * kTile8U4;
        uint4 k[8], v[8];
        load_k8(k, kc + at, lane);
        load_v8(v, vc + at, lane);
        float z[4];
        scores8(z, k, q, lane);
        const float f = score_factor(q.unit, __shfl_sync(0xffffffffu, bl.ks, t), scale_log2);
        const int visible = p - __shfl_sync(0xffffffffu, bl.j, t) * kBlock + 1;   // at least 1
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] *= f;
        if (visible < kBlock) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (8 * i + g >= visible) z[i] = -INFINITY;
            mask_v8(v, visible, lane);
        }
        float mb = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, x));
        mb = fmaxf(mb, kLeast);   // every score -inf: weights 0, not NaN
        const float ahead = st.m - mb, less = exp2_approx(-fabsf(ahead));
        const float corr = ahead > 0.f ? 1.f : less, fresh = ahead > 0.f ? less : 1.f;   // of what was, of the block
        float w[4], lb = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = exp2_approx(z[i] - mb);
            lb += w[i];
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) lb += __shfl_xor_sync(0xffffffffu, lb, x);
        st.m = fmaxf(st.m, mb);
        st.l = fmaf(st.l, corr, lb * fresh);
#pragma unroll
        for (int e = 0; e < 16; ++e) st.acc[e] *= corr;
        weighted_sum8(st.acc, w, v, __shfl_sync(0xffffffffu, bl.vs, t) * fresh, lane);
        done(t, mb, lb);
    }
}

// Warp states, to be merged over a CTA's warps.
template <int kWarps>
struct Merge8 {
    float acc[kWarps][kD];
    float2 ml[kWarps];   // {m, l}
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
// The merged state, by threads d < 128 after a barrier: thread d gets dim d of the output.
template <int kWarps>
__device__ __forceinline__ void merge8(const Merge8<kWarps> &s, int d, float &M, float &L, float &A) {
    float2 ml[kWarps];
    float a[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        ml[w] = s.ml[w];
        a[w] = s.acc[w][d];
    }
    M = ml[0].x;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, ml[w].x);
    const float base = M == -INFINITY ? 0.f : M;
    L = A = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(ml[w].x - base);   // 0 for an empty state
        L = fmaf(ml[w].y, f, L);
        A = fmaf(a[w], f, A);
    }
}

// The page of block j; -1 and a flag when it is outside the pool.
__device__ __forceinline__ int checked_page(const int32_t *bt_row, int j, int num_pages, int32_t *dev_err) {
    const int page = __ldg(bt_row + j);
    if ((unsigned)page < (unsigned)num_pages) return page;
    flag_error(dev_err, UOCR_DEVERR_PAGE);
    return -1;
}

constexpr int kSWarps = 4;       // sparse: warps of a CTA
constexpr int kDWarps = 4;       // dense: warps of a CTA, each every fourth block of its chunk
constexpr int kMergeThreads = 512;

}  // namespace

// A cluster of kCluster CTAs of 4 warps per (query, head); warp w of CTA r attends the selection slots
// 4 r + w, + 4 kCluster, ...  With four CTAs every warp has one block, and the four meet in CTA 0
// through its shared memory: an SM takes in 64 bytes a clock, so the 128 KiB of a (query, head)
// alone keep one for 1 us (10 pairs take 6.9 us with one CTA each, 4.6 with four).  With
// enough pairs to fill the SMs one CTA does all 16.
// kSeq: the queries are a chunk of one sequence.
template <int kCluster, bool kSeq>
__global__ void __launch_bounds__(kSWarps * 32, 5)
sparse_attn_kv8_kernel(const uint2 *__restrict__ q, const uint4 *__restrict__ kc, const uint4 *__restrict__ vc,
                       const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                       const int32_t *__restrict__ bt, const int32_t *__restrict__ seq_lens,
                       const int32_t *__restrict__ q_seq, const int32_t *__restrict__ q_pos,
                       const int32_t *__restrict__ sel, int B, int H, int max_blocks, int num_pages,
                       float scale_log2, int implicit_local, int fixed_seq, __nv_bfloat16 *__restrict__ out,
                       float *__restrict__ mass, unsigned long long *mass_fx, int32_t *dev_err) {
    constexpr int kStep = kSWarps * kCluster, kPer = kSel / kStep;
    __shared__ __align__(16) Merge8<kSWarps> s;
    __shared__ __align__(16) Merge8<kCluster> s_all;   // of CTA 0: the CTAs' states
    __shared__ Query8Smem s_q[kSWarps];
    __shared__ float s_slot[4][kSel];                  // of CTA 0, per slot: m, l, block (as bits), total before
    const int rank = kCluster > 1 ? cluster_rank() : 0;
    if (kCluster > 1) cluster_arrive();
    const int ih = blockIdx.x / kCluster, i = ih / H, h = ih - i * H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = rank * kSWarps + warp + kStep * (lane % kPer);   // of the lanes below kPer

    // the selection, the query and the lengths are on their way before any of them is used
    const int32_t *my_sel = sel + (size_t)i * kSel + slot;
    int j = implicit_local ? -2 : ld_pinned(my_sel);   // with implicit_local, -2: not known yet
    const uint2 raw = __ldg(q + (size_t)ih * (kD / 4) + lane);
    QueryRef r;
    const bool report = threadIdx.x == 0 && h == 0 && rank == 0;
    bool ok = resolve_query(i, seq_lens, q_seq, q_pos, B, max_blocks, dev_err, report, r, kSeq ? fixed_seq : -1);
    if (kSeq && ok && r.p < 0) {   // a chunk's positions are the caller's
        if (report) flag_error(dev_err, UOCR_DEVERR_POS);
        ok = false;
    }
    if (!ok || (!implicit_local && j < 0)) j = -1;   // a caller's slot below 0 is empty, whatever its value
    if (j == -2) {   // after the selection kernel: slots that do not depend on the scores (see sparse_attn.cu)
        if (r.nb <= kSel)
            j = slot < r.nb ? slot : -1;
        else if (slot >= kRemote)
            j = r.nb - kSel + slot;
    }
    if (__any_sync(0xffffffffu, j == -2)) {
        pdl_wait();
        if (j == -2) j = __ldcg(my_sel);
    }
    if (lane >= kPer) j = -1;
    if (j >= 0 && j >= r.nb) {
        flag_error(dev_err, UOCR_DEVERR_SEL);
        j = -1;
    }
    Blocks8 bl;
    bl.page = j >= 0 ? checked_page(bt + (size_t)r.b * max_blocks, j, num_pages, dev_err) : -1;
    const Query8 query = split_query8(s_q[warp], raw, lane);   // while the page is on its way
    bl.j = bl.page >= 0 ? j : -1;
    load_scales8(bl, k_scale, v_scale, H, h);
    float *const totals = !kSeq && mass ? mass + ((size_t)(ok ? r.b : 0) * H + h) * max_blocks : nullptr;
    const float before = totals && bl.j >= 0 ? __ldcg(totals + bl.j) : 0.f;   // in flight beside the attention

    State8 st;
    float2 mine = make_float2(-INFINITY, 0.f);   // of the lane's slot
    attend8(st, bl, kc, vc, H, h, ok ? r.p : -1, scale_log2, query, lane, [&](int t, float m, float l) {
        if (lane == t) mine = make_float2(m, l);
    });
    put_state8(s, st, warp, lane);
    if (kCluster > 1) cluster_wait();   // every CTA of the cluster has started
    if (lane < kPer) {
        const float put[4] = {mine.x, mine.y, __int_as_float(bl.j), before};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (kCluster > 1)
                st_cluster(in_cta(&s_slot[x][slot], 0), put[x]);
            else
                s_slot[x][slot] = put[x];
        }
    }
    __syncthreads();

    const int d = threadIdx.x;   // one of 128
    float M, L, A;
    merge8(s, d, M, L, A);
    if (kCluster > 1) {
        st_cluster(in_cta(&s_all.acc[rank][d], 0), A);
        if (d < 2) st_cluster(in_cta(reinterpret_cast<float *>(&s_all.ml[rank]) + d, 0), d ? L : M);
        cluster_arrive();
        cluster_wait();
        if (rank == 0) merge8(s_all, d, M, L, A);
    }
    if (rank == 0) {
        // L is 0 for a query without a visible token, NaN where a score is
        out[(size_t)ih * kD + d] = __float2bfloat16_rn(L != 0.f ? A / L : 0.f);
        if ((kSeq ? mass_fx != nullptr : totals != nullptr) && warp == 0) {
            // one writer per block: the first slot that names it adds the weights of all that do
            const int x = lane & 15;
            const int block = __float_as_int(s_slot[2][x]);
            float w = s_slot[1][x] * exp2f(s_slot[0][x] - (M == -INFINITY ? 0.f : M));
            const unsigned same = __match_any_sync(0xffffffffu, block) & 0xffffu;
            if (__any_sync(0xffffffffu, block >= 0 && (same & (same - 1)))) {
                float all = 0.f;
                for (int y = 0; y < kSel; ++y) {
                    const float o = __shfl_sync(0xffffffffu, w, y);
                    if (same >> y & 1) all += o;
                }
                w = all;
            }
            if (lane < kSel && block >= 0 && lane == __ffs(same) - 1 && L > 0.f) {
                if (!kSeq)
                    totals[block] = s_slot[3][x] + finite_weight(w / L);
                else   // many queries of one sequence: a sum of integers, in any order
                    atomicAdd(mass_fx + (size_t)h * max_blocks + block, fixed_weight(w / L));
            }
        }
    }
    // warps whose blocks were known in advance did not wait for the selection kernel: this grid
    // still completes after it
    if (blockIdx.x == 0 && threadIdx.x == 0) pdl_wait();
}

// The blocks that a dense query attends, as one list: [0, pre) and [win, nb).
struct Attended {
    int nb, pre, win;
    __device__ __forceinline__ Attended(int causal, int ref_blocks)
        : nb(causal), pre(min(ref_blocks, causal)), win(max(causal - kLocal, min(ref_blocks, causal))) {}
    __device__ __forceinline__ int count() const { return pre + nb - win; }
    __device__ __forceinline__ int block(int t) const { return t < pre ? t : win + t - pre; }
    __device__ __forceinline__ bool has(int j) const { return j < pre || (j >= win && j < nb); }
};

// Split over chunks of the list: CTA (query, head, chunk) leaves {m, l}, acc[128] and, for the
// totals, each block's weight sum with the maximum it refers to.
__global__ void __launch_bounds__(kDWarps * 32, 5)
dense_kv8_chunk_kernel(const uint2 *__restrict__ q, const uint4 *__restrict__ kc, const uint4 *__restrict__ vc,
                       const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                       const int32_t *__restrict__ bt, const int32_t *__restrict__ seq_lens, int B, int H,
                       int max_blocks, int num_pages, int ref_blocks, int chunk_blocks, int n_chunks,
                       float scale_log2, float *__restrict__ part_acc, float2 *__restrict__ part_ml,
                       float2 *__restrict__ blk_ml, int32_t *dev_err) {
    __shared__ __align__(16) Merge8<kDWarps> s;
    __shared__ Query8Smem s_q[kDWarps];
    const int chunk = blockIdx.x % n_chunks, ih = blockIdx.x / n_chunks;
    const int i = ih / H, h = ih - i * H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint2 raw = __ldg(q + (size_t)ih * (kD / 4) + lane);
    QueryRef r;
    const bool ok = resolve_query(i, seq_lens, nullptr, nullptr, B, max_blocks, dev_err,
                                  threadIdx.x == 0 && chunk == 0 && h == 0, r);
    const Attended att(ok ? r.nb : 0, ref_blocks);
    if (chunk * chunk_blocks >= att.count()) return;   // the merge reads only the chunks below that

    const int t = chunk * chunk_blocks + warp + kDWarps * lane;   // of the lanes below chunk_blocks / 4
    const bool mine = lane < chunk_blocks / kDWarps && t < att.count();
    Blocks8 bl;
    bl.j = mine ? att.block(t) : 0;
    bl.page = mine ? checked_page(bt + (size_t)i * max_blocks, bl.j, num_pages, dev_err) : -1;
    const Query8 query = split_query8(s_q[warp], raw, lane);   // while the pages are on their way
    load_scales8(bl, k_scale, v_scale, H, h);
    if (blk_ml && mine && bl.page < 0) blk_ml[(size_t)ih * max_blocks + bl.j] = make_float2(-INFINITY, 0.f);
    State8 st;
    attend8(st, bl, kc, vc, H, h, __ldg(seq_lens + i) - 1, scale_log2, query, lane,
            [&](int t, float m, float l) {
                if (blk_ml && lane == t) blk_ml[(size_t)ih * max_blocks + bl.j] = make_float2(m, l);
            });
    put_state8(s, st, warp, lane);
    __syncthreads();
    const int d = threadIdx.x;
    float M, L, A;
    merge8(s, d, M, L, A);
    const size_t at = (size_t)ih * n_chunks + chunk;
    part_acc[at * kD + d] = A;
    if (d == 0) part_ml[at] = make_float2(M, L);
}

// CTA (query, head, 0) merges the chunks' states into the output, a warp per every sixteenth chunk
// and four dims per lane; CTA (query, head, 1 + x) adds the weights of the blocks [512 x, 512 x + 512)
// to their totals.
__global__ void __launch_bounds__(kMergeThreads)
dense_kv8_merge_kernel(const int32_t *__restrict__ seq_lens, int B, int H, int max_blocks, int ref_blocks,
                       int chunk_blocks, int n_chunks, int parts, const float4 *__restrict__ part_acc,
                       const float2 *__restrict__ part_ml, const float2 *__restrict__ blk_ml, __nv_bfloat16 *__restrict__ out, float *__restrict__ mass) {
    constexpr int kWarps = kMergeThreads / 32;
    __shared__ float s_red[kWarps];
    __shared__ float4 s_acc[kWarps][kD / 4];
    const int ih = blockIdx.x / parts, part = blockIdx.x - ih * parts;
    const int i = ih / H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    QueryRef r;
    const bool ok = resolve_query(i, seq_lens, nullptr, nullptr, B, max_blocks, nullptr, false, r);
    const Attended att(ok ? r.nb : 0, ref_blocks);
    const int used = (att.count() + chunk_blocks - 1) / chunk_blocks;
    if (part > 0 && (part - 1) * kMergeThreads >= att.nb) return;
    const int j = (part - 1) * kMergeThreads + tid;
    const bool add = part > 0 && att.has(j);
    const size_t at = (size_t)ih * max_blocks + j;
    const float before = add ? mass[at] : 0.f;   // not written by the kernel before this one
    pdl_wait();
    const float2 own = add ? __ldcg(blk_ml + at) : make_float2(-INFINITY, 0.f);
    const float2 *ml = part_ml + (size_t)ih * n_chunks;
    // maximum and sum over the chunks, in an order that does not depend on the part
    float2 st = make_float2(-INFINITY, 0.f);
    for (int c = tid; c < used; c += kMergeThreads) {
        const float2 x = __ldcg(ml + c);
        const float m = fmaxf(st.x, x.x), b = m == -INFINITY ? 0.f : m;
        st = make_float2(m, st.y * exp2f(st.x - b) + x.y * exp2f(x.x - b));
    }
    float M = warp_max(st.x);
    if (lane == 0) s_red[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_red[w]);
    __syncthreads();
    const float base = M == -INFINITY ? 0.f : M;
    float L = warp_sum(st.y * exp2f(st.x - base));
    if (lane == 0) s_red[warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L += s_red[w];
    if (part > 0) {
        if (add && L > 0.f) mass[at] = before + finite_weight(own.y * exp2f(own.x - base) / L);
        return;
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = warp; c < used; c += kWarps) {
        const float f = exp2f(__ldcg(ml + c).x - base);
        const float4 v = __ldcg(part_acc + ((size_t)ih * n_chunks + c) * (kD / 4) + lane);
        a.x = fmaf(v.x, f, a.x);
        a.y = fmaf(v.y, f, a.y);
        a.z = fmaf(v.z, f, a.z);
        a.w = fmaf(v.w, f, a.w);
    }
    s_acc[warp][lane] = a;
    __syncthreads();
    if (tid < kD) {
        float A = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) A += reinterpret_cast<const float *>(s_acc[w])[tid];
        out[(size_t)ih * kD + tid] = __float2bfloat16_rn(L != 0.f ? A / L : 0.f);
    }
}

// ------------------------------------------------------------------ host side
cudaError_t launch_sparse_attn_kv8(const LaunchCtx &c, const void *q, const Kv8Cache &kv, const int32_t *bt,
                                   const int32_t *seq_lens, const int32_t *q_seq, const int32_t *q_pos,
                                   const int32_t *sel, int n_q, int B, int H, int max_blocks, int num_pages,
                                   float scale, void *out, float *mass, bool implicit_local, int32_t *dev_err,
                                   int fixed_seq, unsigned long long *mass_fx) {
    const long long grid = (long long)n_q * H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    // As many CTAs per pair as can all be resident at once, 5 a SM; clusters of 4 do not fill every GPC to
    // its last slot (176 pairs no longer fit on 148 SMs, and how many do depends on the GPCs), so for them
    // 4.5.  Measured with 1 / 2 / 4 (us; 148 SMs): 10 pairs 6.9 / 5.7 / 4.6, 140: 10.5 / 8.3 / 7.6, 160: 10.9 /
    // 8.7 / 8.3, 175: 11.1 / 8.8 / 8.3, 176: 11.0 / 8.7 / 11.0, 300: 12.2 / 11.5 / 14.9, 370: 13.5 / 13.1 /
    // 19.2, 450: 14.9 / 19.1 / 21.1.
    const int cluster = 8 * grid <= 9 * c.num_sms ? 4 : 2 * grid <= 5 * c.num_sms ? 2 : 1;
    attr[0].val.clusterDim.x = cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cluster * grid));
    cfg.blockDim = dim3(kSWarps * 32);
    cfg.stream = c.stream;
    cfg.attrs = cluster > 1 ? attr : attr + 1;
    cfg.numAttrs = (cluster > 1 ? 1 : 0) + (c.pdl ? 1 : 0);
    auto pick = [cluster](auto four, auto two, auto one) { return cluster == 4 ? four : cluster == 2 ? two : one; };
    auto kernel = fixed_seq >= 0 ? pick(sparse_attn_kv8_kernel<4, true>, sparse_attn_kv8_kernel<2, true>,
                                        sparse_attn_kv8_kernel<1, true>)
                                 : pick(sparse_attn_kv8_kernel<4, false>, sparse_attn_kv8_kernel<2, false>,
                                        sparse_attn_kv8_kernel<1, false>);
    return cudaLaunchKernelEx(&cfg, kernel, (const uint2 *)q, (const uint4 *)kv.k, (const uint4 *)kv.v, kv.k_scale,
                              kv.v_scale, bt, seq_lens, q_seq, q_pos, sel, B, H, max_blocks, num_pages,
                              scale * kLog2e, implicit_local ? 1 : 0, fixed_seq, (__nv_bfloat16 *)out, mass, mass_fx,
                              dev_err);
}

namespace {
struct Dense8Ws {
    int chunk_blocks, n_chunks;
    size_t acc_off, ml_off, blk_off, total;
};
// Blocks of a chunk, by the CTAs that would come of it where every row attends all that it may: the
// shortest whose CTAs are all resident at once (740 on 148 SMs), for more warps on the same bytes; past
// that 16, for fewer prologues and partial states.  32 blocks only for one sequence: where several
// differ in length, the longest one's last CTAs then run alone.  Measured (us, 10 heads) with 4 / 8 / 16 / 32
// blocks: 1 x 16384 tokens 17.2 / 14.7 / 14.0 / -; 5 x <= 9001 with a prefix of 100 blocks 14.1 / 13.2 /
// 14.7 / -; 1 x 60000 with one of 20 6.2 / - / 12.4 / -; 4 x 8192 - / 21.2 / 19.4 / -; 16 x 4096 - / 35.7 / 34.1 / -;
// 1 x 131072 - / 64.9 / 61.9 / 59.9; 16 x 32768 - / - / 209 / 207; 40 x 500 .. 12000 - / - / 107 / 111;
// 3 x 100 .. 60000 - / 48.1 / 46.5 / 50.9.
constexpr size_t kResident = 740;
int dense8_chunk(int n_q, int H, int blocks) {
    auto ctas = [&](int chunk) { return (size_t)n_q * H * ((blocks + chunk - 1) / chunk); };
    if (n_q == 1 && ctas(32) >= kResident) return 32;
    return ctas(4) <= kResident ? 4 : ctas(8) <= kResident ? 8 : 16;
}
Dense8Ws dense8_layout(int n_q, int H, int max_blocks, int ref_blocks) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Dense8Ws w{};
    const size_t rows = (size_t)n_q * H;
    const int blocks = (int)min((long long)max_blocks, (long long)ref_blocks + kLocal);
    w.chunk_blocks = dense8_chunk(n_q, H, blocks);
    w.n_chunks = (blocks + w.chunk_blocks - 1) / w.chunk_blocks;
    // chunks below 16 blocks are taken for kResident CTAs at most: the workspace holds any ref_blocks
    const size_t slots = max(rows * ((max_blocks + 15) / 16), kResident);
    w.ml_off = up(slots * kD * 4);
    w.blk_off = w.ml_off + up(slots * sizeof(float2));
    w.total = w.blk_off + up(rows * max_blocks * sizeof(float2));
    return w;
}
}  // namespace

size_t dense_kv8_workspace(int n_q, int H, int max_blocks) { return dense8_layout(n_q, H, max_blocks, 0).total; }

cudaError_t launch_dense_kv8(const LaunchCtx &c, const void *q, const Kv8Cache &kv, const int32_t *bt,
                             const int32_t *seq_lens, int B, int H, int max_blocks, int num_pages, int ref_blocks,
                             float scale, void *out, float *mass, void *ws, int32_t *dev_err) {
    const Dense8Ws w = dense8_layout(B, H, max_blocks, ref_blocks);
    float *acc = (float *)((char *)ws + w.acc_off);
    float2 *ml = (float2 *)((char *)ws + w.ml_off);
    float2 *blk = mass ? (float2 *)((char *)ws + w.blk_off) : nullptr;
    const long long grid = (long long)B * H * w.n_chunks;
    const int parts = mass ? 1 + (max_blocks + kMergeThreads - 1) / kMergeThreads : 1;
    if (grid > 0x7fffffffLL || (long long)B * H * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kDWarps * 32);
    cfg.stream = c.stream;
    cudaError_t e = cudaLaunchKernelEx(&cfg, dense_kv8_chunk_kernel, (const uint2 *)q, (const uint4 *)kv.k,
                                       (const uint4 *)kv.v, kv.k_scale, kv.v_scale, bt, seq_lens, B, H, max_blocks,
                                       num_pages, ref_blocks, w.chunk_blocks, w.n_chunks, scale * kLog2e, acc, ml, blk,
                                       dev_err);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(B * H * parts));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dense_kv8_merge_kernel, seq_lens, B, H, max_blocks, ref_blocks,
                              w.chunk_blocks, w.n_chunks, parts, (const float4 *)acc, (const float2 *)ml,
                              (const float2 *)blk, (__nv_bfloat16 *)out, mass);
}

}  // namespace uocr
