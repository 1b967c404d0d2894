// kv8_prefill.cu -- attention of many queries of one sequence, each over its own 16 selected
// blocks, from a key / value cache held in e4m3 with a scale for each (page, head).
//
// The result of sparse_attn_kv8 for every query (Unlimited-OCR-2 walk-through,
// news.rkmt.cn/news/25027, section 五 step 4), computed block by block as the bf16 form does
// (prefill_attn.cu), so that a (block, head) tile is read once for all the queries that chose it:
//   1. prepare   a CTA per query: its selection is checked and counted per block, and its rows are
//                turned into fp16, in the order in which the products load them, each row times a
//                power of two that brings its largest element to 2^14 (exact, see kv8.cuh);
//   2. invert    per block, the list of the (query, slot) entries that chose it, in items of at
//                most 16 (the bf16 form's kernel);
//   3. blocks    one warp per (item, head): S = Q K8^T (16 x 32), an fp32 softmax per row,
//                P V8 (16 x 128); leaves each entry's maximum, weight sum and the block's value scale
//                in fp32 and its unnormalised output in fp16;
//   4. merge     half a warp per (query, head): out = sum_k 2^(m_k - M) vs_k acc_k / L,
//                L = sum_k 2^(m_k - M) l_k; with totals asked for, the weight 2^(m_k - M) l_k / L of
//                each slot is added to its block's as a multiple of 2^-40 (integers: the sum does
//                not depend on the order of the atomics);
//   5. totals    the sums of step 4 added to the running totals.
// Roundings to fewer than 32 bits: the weights p in [0, 1] to fp16 for P V (2^-11 relative, their
// sum l keeps 32 bits) and the partial outputs to fp16 (2^-11; |acc| <= 32 * 448, in units of the
// block's value scale, so fp16 holds it): each an eighth of the output's own rounding to bf16.
//
// Staging of step 3.  A lane's operand registers are whole 16-byte pieces of K, V and Q rows, so each
// lane copies its own 24 pieces into its own place in shared memory with cp.async and reads them
// back: no lane reads what another wrote, so there is no barrier, no swizzle and no bank conflict,
// only a queue that costs no registers.  The next unit's K and Q start once this unit's S is done, its
// V once P V is; its entries are loaded one unit ahead and its record two, so that a unit waits for
// one memory latency at most.
#include <math.h>

#include "kernels.h"
#include "kv8.cuh"

namespace uocr {

namespace {
constexpr int kRows = 16;        // entries of an item
constexpr int kBlkWarps = 4, kBlkCtas = 4;
constexpr int kMrgWarps = 8;
constexpr float kMassUnit = 1.f / (1ll << 40);

// A warp's queue: piece x of lane l at x * 32 + l.
struct UnitSmem {
    uint4 k[8 * 32], v[8 * 32], q[8 * 32];
};

// Four codes to fp16 where it stands in the program: moved ahead, the conversions of a whole tile
// would hold 64 registers.
__device__ __forceinline__ void to_f16_here(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm volatile("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
                 : "=r"(lo), "=r"(hi)
                 : "r"(v));
}
template <int kDst>
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint4 *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + kDst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
// Stores that stay in L2 for the merge of the same call.
__device__ __forceinline__ void st_keep(uint4 *p, const uint4 &v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void discard_line(const void *p) {   // 128 bytes, not written back
    asm volatile("discard.global.L2 [%0], 128;" ::"l"(p) : "memory");
}
}  // namespace

// q16 [n_q][H][16] pieces of 8 dims: piece 4 x + c holds dims 64 (x / 2) + 16 c + 8 (x % 2) .. + 7.
__global__ void __launch_bounds__(128)
kv8_prepare_kernel(const uint4 *__restrict__ q, const int32_t *__restrict__ sel, const int32_t *__restrict__ q_pos,
                   const int32_t *__restrict__ seq_len_ptr, int H, int max_blocks, int32_t *__restrict__ sel_ws,
                   int32_t *counts, uint4 *__restrict__ q16, float *__restrict__ unit, int32_t *dev_err) {
    const int i = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    if (tid < kSel) {
        const int len = __ldg(seq_len_ptr), p = __ldg(q_pos + i);
        const bool ok = p >= 0 && p < len && len <= max_blocks * kBlock;
        if (!ok && tid == 0) flag_error(dev_err, UOCR_DEVERR_POS);
        int j = ok ? __ldcg(sel + (size_t)i * kSel + tid) : -1;
        if (j > p / kBlock) {
            flag_error(dev_err, UOCR_DEVERR_SEL);
            j = -1;
        }
        if (j < 0) j = -1;
        sel_ws[(size_t)i * kSel + tid] = j;
        if (j >= 0) atomicAdd(counts + j, 1);
    }
    // 16 lanes per (query, head) row, 8 dims each
    const int l = tid & 15;
    for (int h0 = 0; h0 < H; h0 += 8) {
        const int h = h0 + (tid >> 4);
        const bool live = h < H;
        float x[8];
        float amax = 0.f;
        bf16x8_to_f32(live ? __ldg(q + ((size_t)i * H + h) * 16 + l) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float inv;
        const float s = f16_row_scale(amax, inv);
        if (live) {
            // dims 8 l ..: half l / 8, c = (l % 8) / 2, x % 2 = l % 2
            const int piece = 4 * (2 * (l >> 3) + (l & 1)) + ((l & 7) >> 1);
            q16[((size_t)i * H + h) * 16 + piece] =
                make_uint4(pack_f16(x[0] * s, x[1] * s), pack_f16(x[2] * s, x[3] * s), pack_f16(x[4] * s, x[5] * s),
                           pack_f16(x[6] * s, x[7] * s));
            if (l == 0) unit[(size_t)i * H + h] = inv;
        }
    }
}

__global__ void __launch_bounds__(kBlkWarps * 32, kBlkCtas)
kv8_block_kernel(const uint4 *__restrict__ q16, const float *__restrict__ unit, const uint4 *__restrict__ kc,
                 const uint4 *__restrict__ vc, const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                 const int2 *__restrict__ list, const int4 *__restrict__ items, const int32_t *__restrict__ n_items,
                 int H, int num_pages, float scale_log2, uint4 *__restrict__ part_o, float4 *__restrict__ part_ml,
                 int32_t *dev_err) {
    __shared__ UnitSmem sm[kBlkWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint4 *sk = sm[warp].k + lane, *sv = sm[warp].v + lane, *sq = sm[warp].q + lane;
    const uint32_t ak = smem_addr(sk), av = smem_addr(sv), aq = smem_addr(sq);
    uint64_t keep;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    pdl_wait();

    // Units (item, head), heads innermost, dealt round-robin over the warps: unit u is (item, h), the
    // warp's next one (item + d_item, h + d_h) with a carry.
    const int count = __ldcg(n_items);
    const int step = gridDim.x * kBlkWarps, d_item = step / H, d_h = step - d_item * H;
    struct Place {
        int item, h;
    };
    auto advance = [&](Place u) {
        u.item += d_item;
        u.h += d_h;
        if (u.h >= H) {
            u.h -= H;
            ++u.item;
        }
        return u;
    };
    auto load_rec = [&](const Place &u) {   // {block, page, first entry, entries}; no entries past the end
        return u.item < count ? __ldcg(items + u.item) : make_int4(0, -1, 0, 0);
    };
    // rows past the item's end repeat its last entry and store nothing
    auto load_entry = [&](const int4 &rec, int row) {   // {query * 16 + slot, position}
        return rec.w > 0 ? __ldcg(list + rec.z + min(row, rec.w - 1)) : make_int2(0, 0);
    };
    auto page_ok = [&](const int4 &rec) { return (unsigned)rec.y < (unsigned)num_pages; };
    auto issue_qk = [&](const int4 &rec, int h, int2 ea, int2 eb) {
        if (page_ok(rec)) {
            const uint4 *src = kc + ((size_t)rec.y * H + h) * kTile8U4 + g * kRowU4 + c;
            cp_async16<0 * 512>(ak, src);
            cp_async16<1 * 512>(ak, src + 4);
            cp_async16<2 * 512>(ak, src + 8 * kRowU4);
            cp_async16<3 * 512>(ak, src + 8 * kRowU4 + 4);
            cp_async16<4 * 512>(ak, src + 16 * kRowU4);
            cp_async16<5 * 512>(ak, src + 16 * kRowU4 + 4);
            cp_async16<6 * 512>(ak, src + 24 * kRowU4);
            cp_async16<7 * 512>(ak, src + 24 * kRowU4 + 4);
            // rows g and g + 8
            const uint4 *qa = q16 + ((size_t)(ea.x >> 4) * H + h) * 16 + c;
            const uint4 *qb = q16 + ((size_t)(eb.x >> 4) * H + h) * 16 + c;
            cp_async16<0 * 512>(aq, qa);
            cp_async16<1 * 512>(aq, qa + 4);
            cp_async16<2 * 512>(aq, qa + 8);
            cp_async16<3 * 512>(aq, qa + 12);
            cp_async16<4 * 512>(aq, qb);
            cp_async16<5 * 512>(aq, qb + 4);
            cp_async16<6 * 512>(aq, qb + 8);
            cp_async16<7 * 512>(aq, qb + 12);
        }
        cp_commit();
    };
    // v piece 4 s + j: piece g of token 16 s + 8 (j / 2) + 2 c + j % 2, so that P's accumulator layout is
    // the operand's
    auto issue_v = [&](const int4 &rec, int h) {
        if (page_ok(rec)) {
            const uint4 *src = vc + ((size_t)rec.y * H + h) * kTile8U4 + 2 * c * kRowU4 + g;
            cp_async16<0 * 512>(av, src);
            cp_async16<1 * 512>(av, src + kRowU4);
            cp_async16<2 * 512>(av, src + 8 * kRowU4);
            cp_async16<3 * 512>(av, src + 9 * kRowU4);
            cp_async16<4 * 512>(av, src + 16 * kRowU4);
            cp_async16<5 * 512>(av, src + 17 * kRowU4);
            cp_async16<6 * 512>(av, src + 24 * kRowU4);
            cp_async16<7 * 512>(av, src + 25 * kRowU4);
        }
        cp_commit();
    };

    const int first = blockIdx.x * kBlkWarps + warp;
    Place at{first / H, first % H};
    int4 rec = load_rec(at);
    int2 ea = load_entry(rec, g), eb = load_entry(rec, g + 8);
    issue_qk(rec, at.h, ea, eb);
    issue_v(rec, at.h);
    Place at1 = advance(at);
    int4 rec1 = load_rec(at1);
    int2 ea1 = load_entry(rec1, g), eb1 = load_entry(rec1, g + 8);
    Place at2 = advance(at1);
    int4 rec2 = load_rec(at2);

    while (rec.w > 0) {
        const int h = at.h;
        const int row_a = (ea.x >> 4) * H + h, row_b = (eb.x >> 4) * H + h;   // below 2^30
        const bool good = page_ok(rec);
        float vs = 0.f, ks = 0.f, ua = 0.f, ub = 0.f;
        if (good) {
            const size_t tile = (size_t)rec.y * H + h;
            ks = __ldg(k_scale + tile);
            vs = __ldg(v_scale + tile);
            ua = __ldcg(unit + row_a);
            ub = __ldcg(unit + row_b);
        } else if (lane == 0) {
            flag_error(dev_err, UOCR_DEVERR_PAGE);
        }

        // ---- S: rows g, g + 8; tokens 8 nt + 2 c, + 1
        cp_wait<1>();
        float s[4][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            uint4 k[4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) k[nt] = sk[32 * (2 * nt + f)];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint4 a = sq[32 * (2 * f + y)], b = sq[32 * (4 + 2 * f + y)];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    uint32_t b0, b1;
                    to_f16_here(y ? k[nt].z : k[nt].x, b0, b1);
                    if (f == 0 && y == 0)
                        mma_f16_new(s[nt], a.x, b.x, a.y, b.y, b0, b1);
                    else
                        mma_f16(s[nt], a.x, b.x, a.y, b.y, b0, b1);
                    to_f16_here(y ? k[nt].w : k[nt].y, b0, b1);
                    mma_f16(s[nt], a.z, b.z, a.w, b.w, b0, b1);
                }
            }
        }
        issue_qk(rec1, at1.h, ea1, eb1);   // K and Q are in registers or used

        // ---- causal mask, maxima, weights
        const int t0 = rec.x * kBlock;
        const int far = __reduce_max_sync(0xffffffffu, max(ea.y, eb.y)) - t0 + 1;
        const int near = __reduce_min_sync(0xffffffffu, min(ea.y, eb.y)) - t0 + 1;
        ks *= scale_log2;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[nt][e] = s[nt][e] * ua * ks;
                s[nt][2 + e] = s[nt][2 + e] * ub * ks;
            }
        if (near < kBlock) {   // some query does not see the whole block
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tok = t0 + 8 * nt + 2 * c + e;
                    if (tok > ea.y) s[nt][e] = -INFINITY;
                    if (tok > eb.y) s[nt][2 + e] = -INFINITY;
                }
        }
        float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ma = fmaxf(ma, s[nt][e]);
                mb = fmaxf(mb, s[nt][2 + e]);
            }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, x));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, x));
        }
        const float base_a = ma == -INFINITY ? 0.f : ma, base_b = mb == -INFINITY ? 0.f : mb;
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            const float p0 = exp2_approx(s[nt][0] - base_a), p1 = exp2_approx(s[nt][1] - base_a);
            const float p2 = exp2_approx(s[nt][2] - base_b), p3 = exp2_approx(s[nt][3] - base_b);
            la += p0 + p1;
            lb += p2 + p3;
            pa[nt] = pack_f16(p0, p1);
            pb[nt] = pack_f16(p2, p3);
        }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            la += __shfl_xor_sync(0xffffffffu, la, x);
            lb += __shfl_xor_sync(0xffffffffu, lb, x);
        }

        // ---- O = P V8: rows g, g + 8; column n of MMA e is dim 16 n + e
        cp_wait<1>();
        auto v_token = [&](int x) { return 16 * (x >> 2) + 8 * ((x >> 1) & 1) + 2 * c + (x & 1); };
        // A token behind a query's position has weight 0, but 0 * NaN is not 0.  Tokens that no query
        // of the item sees may hold anything and are cut off for all of them; where some queries see
        // a token that others do not and its value is NaN, each row gets a product of its own.
        bool apart = false;
        if (near < min(far, kBlock)) {
            uint32_t nan = 0u;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint4 v = sv[32 * x];
                if (v_token(x) < far)
#pragma unroll
                    for (int w = 0; w < 4; ++w) nan |= __vcmpeq4(word(v, w) & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
            apart = __any_sync(0xffffffffu, nan != 0u);
        }
#pragma unroll 1
        for (int turn = 0; turn < (apart ? kRows : 1); ++turn) {
            int seen = far;
            bool want_a = g < rec.w, want_b = g + 8 < rec.w;
            if (apart) {
                seen = __shfl_sync(0xffffffffu, turn < 8 ? ea.y : eb.y, 4 * (turn & 7)) - t0 + 1;
                want_a = want_a && turn == g;
                want_b = want_b && turn == g + 8;
            }
            uint32_t oa[2][8], ob[2][8];   // fp16 pairs of dims 32 c + 16 half + 2 i, + 1
            uint4 v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = sv[32 * x];
            if (seen < kBlock) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (v_token(x) >= seen) v[x] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) {
                float o[4][4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t b0[4], b1[4];
                    const uint32_t t0w = word(v[4 * kk], w4), t1w = word(v[4 * kk + 1], w4);
                    const uint32_t t2w = word(v[4 * kk + 2], w4), t3w = word(v[4 * kk + 3], w4);
                    to_f16_here(__byte_perm(t0w, t1w, 0x5140), b0[0], b0[1]);
                    to_f16_here(__byte_perm(t0w, t1w, 0x7362), b0[2], b0[3]);
                    to_f16_here(__byte_perm(t2w, t3w, 0x5140), b1[0], b1[1]);
                    to_f16_here(__byte_perm(t2w, t3w, 0x7362), b1[2], b1[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kk == 0)
                            mma_f16_new(o[e], pa[0], pb[0], pa[1], pb[1], b0[e], b1[e]);
                        else
                            mma_f16(o[e], pa[2], pb[2], pa[3], pb[3], b0[e], b1[e]);
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        oa[half][2 * w4 + e] = pack_f16(o[2 * e][half], o[2 * e + 1][half]);
                        ob[half][2 * w4 + e] = pack_f16(o[2 * e][2 + half], o[2 * e + 1][2 + half]);
                    }
            }
            if (want_a) {
                uint4 *dst = part_o + ((size_t)row_a * kSel + (ea.x & 15)) * 16 + 4 * c;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    st_keep(dst + x, make_uint4(oa[x >> 1][4 * (x & 1)], oa[x >> 1][4 * (x & 1) + 1],
                                                oa[x >> 1][4 * (x & 1) + 2], oa[x >> 1][4 * (x & 1) + 3]), keep);
            }
            if (want_b) {
                uint4 *dst = part_o + ((size_t)row_b * kSel + (eb.x & 15)) * 16 + 4 * c;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    st_keep(dst + x, make_uint4(ob[x >> 1][4 * (x & 1)], ob[x >> 1][4 * (x & 1) + 1],
                                                ob[x >> 1][4 * (x & 1) + 2], ob[x >> 1][4 * (x & 1) + 3]), keep);
            }
        }
        issue_v(rec1, at1.h);   // V is in registers or used

        if (c == 0) {   // (a page outside the pool: nothing was copied, the state is empty)
            if (g < rec.w)
                part_ml[(size_t)row_a * kSel + (ea.x & 15)] = make_float4(good ? ma : -INFINITY, good ? la : 0.f, vs, 0.f);
            if (g + 8 < rec.w)
                part_ml[(size_t)row_b * kSel + (eb.x & 15)] = make_float4(good ? mb : -INFINITY, good ? lb : 0.f, vs, 0.f);
        }
        at = at1;
        rec = rec1;
        ea = ea1;
        eb = eb1;
        at1 = at2;
        rec1 = rec2;
        ea1 = load_entry(rec1, g);
        eb1 = load_entry(rec1, g + 8);
        at2 = advance(at2);
        rec2 = load_rec(at2);
    }
    cp_wait<0>();
}

__global__ void __launch_bounds__(kMrgWarps * 32)
kv8_merge_kernel(const int32_t *__restrict__ sel_ws, const uint4 *__restrict__ part_o,
                 const float4 *__restrict__ part_ml, int n_rows, int H, int max_blocks, uint4 *__restrict__ out,
                 unsigned long long *mass_fx) {
    const int k = threadIdx.x & 15;
    const int row = (blockIdx.x * kMrgWarps * 32 + threadIdx.x) >> 4;
    pdl_wait();
    const bool live = row < n_rows;
    const int ih = live ? row : n_rows - 1;   // every lane takes part in the shuffles
    const int i = ih / H, h = ih - i * H;
    const int j = live ? __ldcg(sel_ws + (size_t)i * kSel + k) : -1;
    const size_t slot = (size_t)ih * kSel;
    const float4 ml = j >= 0 ? __ldcg(part_ml + slot + k) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    float M = ml.x;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    // an empty state's output is not read: it may be anything (a state of NaN scores has a NaN sum)
    const bool some = ml.x != -INFINITY || ml.y != 0.f;
    const float f = exp2f(ml.x - (M == -INFINITY ? 0.f : M));
    const float w = ml.y * f;
    float L = w;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float fv = f * ml.z;
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = 0.f;
    uint4 v[kSel];
#pragma unroll
    for (int s = 0; s < kSel; ++s) {
        const bool has = __shfl_sync(0xffffffffu, (int)some, s, 16);
        v[s] = has ? __ldcg(part_o + (slot + s) * 16 + k) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int s = 0; s < kSel; ++s) {
        const float fs = __shfl_sync(0xffffffffu, fv, s, 16);
        const uint32_t u[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&u[e]));
            a[2 * e] = fmaf(fs, y.x, a[2 * e]);
            a[2 * e + 1] = fmaf(fs, y.y, a[2 * e + 1]);
        }
    }
    __syncwarp();   // every lane of the row has its values
    if (!live) return;
    // this row's partials are read: their lines need not be written back (the workspace is aligned
    // to 256 bytes, so 16 x 256 bytes of outputs are 32 lines of their own and the states two)
    {
        const char *po = reinterpret_cast<const char *>(part_o + slot * 16);
        discard_line(po + 256 * k);
        discard_line(po + 256 * k + 128);
        if (k < 2) discard_line(reinterpret_cast<const char *>(part_ml + slot) + 128 * k);
    }
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 y = L != 0.f ? __floats2bfloat162_rn(a[2 * e] / L, a[2 * e + 1] / L)
                                                : __floats2bfloat162_rn(0.f, 0.f);
        r[e] = *reinterpret_cast<const uint32_t *>(&y);
    }
    out[(size_t)ih * 16 + k] = make_uint4(r[0], r[1], r[2], r[3]);
    if (mass_fx && some) {
        const float share = finite_weight(w / L);   // in [0, 1]
        atomicAdd(mass_fx + (size_t)h * max_blocks + j, (unsigned long long)__float2ull_rn(share / kMassUnit));
    }
}

__global__ void __launch_bounds__(256)
kv8_totals_kernel(const unsigned long long *mass_fx, int n, float *mass) {
    const int x = blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    if (x >= n) return;
    const unsigned long long v = __ldcg(mass_fx + x);
    if (v) mass[x] += (float)((double)v * (double)kMassUnit);
}

// ------------------------------------------------------------------ host side
namespace {
struct Kv8PrefillWs {
    size_t counts_off, fill_off, sched_off, mass_off, zero_bytes, n_items_off, items_off, list_off, sel_off, q_off,
        unit_off, ml_off, o_off, total;
};
Kv8PrefillWs layout(int n_q, int H, int max_blocks) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Kv8PrefillWs w{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up(bytes);
        return at;
    };
    w.counts_off = take((size_t)max_blocks * 4);
    w.fill_off = take((size_t)max_blocks * 4);
    w.sched_off = take(4);
    w.mass_off = take((size_t)H * max_blocks * 8);
    w.zero_bytes = off;
    w.n_items_off = take(4);
    w.items_off = take(prefill_item_bound(n_q, max_blocks) * sizeof(int4));
    w.list_off = take((size_t)n_q * kSel * sizeof(int2));
    w.sel_off = take((size_t)n_q * kSel * 4);
    w.q_off = take((size_t)n_q * H * kD * 2);
    w.unit_off = take((size_t)n_q * H * 4);
    w.ml_off = take((size_t)n_q * H * kSel * sizeof(float4));
    w.o_off = take((size_t)n_q * H * kSel * kD * 2);
    w.total = off;
    return w;
}
}  // namespace

size_t prefill_kv8_workspace(int n_q, int H, int max_blocks) { return layout(n_q, H, max_blocks).total; }

cudaError_t zero_prefill_kv8(const LaunchCtx &c, void *ws, int n_q, int H, int max_blocks, int32_t **sched) {
    const Kv8PrefillWs w = layout(n_q, H, max_blocks);
    if (sched) *sched = (int32_t *)((char *)ws + w.sched_off);
    return cudaMemsetAsync(ws, 0, w.zero_bytes, c.stream);
}

cudaError_t launch_prefill_kv8(const LaunchCtx &c, const void *q, const Kv8Cache &kv, const int32_t *bt_row,
                               const int32_t *seq_len_ptr, const int32_t *q_pos, const int32_t *sel, int n_q, int H,
                               int max_blocks, int num_pages, float scale, void *out, float *mass_row, void *ws,
                               int32_t *dev_err) {
    const Kv8PrefillWs w = layout(n_q, H, max_blocks);
    char *base = (char *)ws;
    int32_t *counts = (int32_t *)(base + w.counts_off), *n_items = (int32_t *)(base + w.n_items_off);
    int32_t *sel_ws = (int32_t *)(base + w.sel_off);
    int4 *items = (int4 *)(base + w.items_off);
    int2 *list = (int2 *)(base + w.list_off);
    uint4 *q16 = (uint4 *)(base + w.q_off), *part_o = (uint4 *)(base + w.o_off);
    float *unit = (float *)(base + w.unit_off);
    float4 *ml = (float4 *)(base + w.ml_off);
    unsigned long long *mass_fx = mass_row ? (unsigned long long *)(base + w.mass_off) : nullptr;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = c.pdl ? 1 : 0;
    cfg.gridDim = dim3((unsigned)n_q);
    cfg.blockDim = dim3(128);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_prepare_kernel, (const uint4 *)q, sel, q_pos, seq_len_ptr, H,
                                       max_blocks, sel_ws, counts, q16, unit, dev_err);
    if (e != cudaSuccess) return e;
    e = launch_prefill_invert(c, counts, bt_row, sel_ws, q_pos, n_q, max_blocks, (int32_t *)(base + w.fill_off), items,
                              n_items, list);
    if (e != cudaSuccess) return e;

    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(kBlkCtas * c.num_sms));
    cfg.blockDim = dim3(kBlkWarps * 32);
    e = cudaLaunchKernelEx(&cfg, kv8_block_kernel, (const uint4 *)q16, (const float *)unit, (const uint4 *)kv.k,
                           (const uint4 *)kv.v, kv.k_scale, kv.v_scale, (const int2 *)list, (const int4 *)items,
                           (const int32_t *)n_items, H, num_pages, scale * kLog2e, part_o, ml, dev_err);
    if (e != cudaSuccess) return e;

    const long long rows = (long long)n_q * H;
    cfg.gridDim = dim3((unsigned)((rows + 2 * kMrgWarps - 1) / (2 * kMrgWarps)));
    cfg.blockDim = dim3(kMrgWarps * 32);
    e = cudaLaunchKernelEx(&cfg, kv8_merge_kernel, (const int32_t *)sel_ws, (const uint4 *)part_o, (const float4 *)ml,
                           (int)rows, H, max_blocks, (uint4 *)out, mass_fx);
    if (e != cudaSuccess || !mass_row) return e;
    const int n = H * max_blocks;
    cfg.gridDim = dim3((unsigned)((n + 255) / 256));
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, kv8_totals_kernel, (const unsigned long long *)mass_fx, n, mass_row);
}

}  // namespace uocr
