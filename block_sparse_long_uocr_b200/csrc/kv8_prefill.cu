// kv8_prefill.cu -- attention of many queries of one sequence, each over its own 16 selected
// blocks, from a key / value cache held in e4m3 with a scale for each (page, head).
//
// The result of sparse_attn_kv8 for every query (Unlimited-OCR-2 walk-through,
// news.rkmt.cn/news/25027, section 五 step 4), computed block by block as the bf16 form does
// (prefill_attn.cu), so that a (block, head) tile is read once for all the queries that chose it:
//   1. prepare   the selections are checked and counted per block, and the queries' rows turned into
//                fp16, in the order in which the products load them, each row times a power of two
//                that brings its largest element to 2^14 (exact, see kv8.cuh);
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
// A few queries are attended one by one instead (sparse_attn_kv8_kernel); their weights go the same way.
// Roundings to fewer than 32 bits: the weights p in [0, 1] to fp16 for P V (2^-11 relative, 2^-25 of the
// block's largest at the least; their sum l keeps 32 bits) and the partial outputs to fp16 (2^-11; |acc| <= 32 * 448, in units of the
// block's value scale, so fp16 holds it): each an eighth of the output's own rounding to bf16.
//
// Staging of step 3, per warp: a K tile and a V tile by TMA in the 128-byte swizzle (16-byte piece p
// of row r at p ^ (r & 7)), and the item's query rows by one bulk copy each, 320 bytes apart.  The next
// unit's K and Q start once this unit's S is done, its V once P V is; its entries are loaded one unit
// ahead and its record two, so that a unit waits for one memory latency at most.  Bank conflicts: an
// 8-lane phase of a 16-byte read covers two MMA columns (or rows) g = 2 m, 2 m + 1 and four pieces, so
// column g of K stands for token rho(g) = 4 (g & 1) + g / 2 of its 8 (the two rows then differ in bit 2
// of the swizzle), V's rows c + 4 y are read in the order y ^ (c & 1), put right by the selector of the
// byte permute that pairs them, and neighbouring query rows start 64 bytes of banks apart.
#include <math.h>
#include <stddef.h>

#include "kernels.h"
#include "kv8.cuh"

namespace uocr {

namespace {
constexpr int kRows = 16;        // entries of an item
constexpr int kBlkWarps = 4, kBlkCtas = 4;
constexpr int kMrgWarps = 8;

constexpr int kQStride = kD * 2 + 64;

struct __align__(1024) UnitSmem {
    uint8_t k[kTile8], v[kTile8];
    uint8_t q[kRows * kQStride];
};

// Four codes to fp16 where it stands in the program: moved ahead, the conversions of a whole tile
// would hold 64 registers.
__device__ __forceinline__ void to_f16_here(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm volatile("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
                 : "=r"(lo), "=r"(hi)
                 : "r"(v));
}
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap *map, int tile, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %2, "
        "%3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(tile), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void bulk_row(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ uint4 ld_smem(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// Stores that stay in L2 for the merge of the same call.
__device__ __forceinline__ void st_keep(uint4 *p, const uint4 &v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w), "l"(policy)
                 : "memory");
}
// A load that is issued where it stands, so that a row's 16 are in flight together.
__device__ __forceinline__ uint4 ld_l2(const uint4 *p, bool wanted) {   // zeros where not wanted
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    asm volatile(
        "{\n .reg .pred w;\n setp.ne.s32 w, %5, 0;\n @w ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];\n}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((int)wanted)
        : "memory");
    return v;
}
__device__ __forceinline__ void discard_line(const void *p) {   // 128 bytes, not written back
    asm volatile("discard.global.L2 [%0], 128;" ::"l"(p) : "memory");
}
}  // namespace

// q16 [n_q][H][16] pieces of 8 dims: piece 4 x + c holds dims 64 (x / 2) + 16 c + 8 (x % 2) .. + 7.
// The first CTAs take 16 (query, head) rows each, 16 lanes a row; the others 16 queries' selections.
__global__ void __launch_bounds__(256)
kv8_prepare_kernel(const uint4 *__restrict__ q, const int32_t *__restrict__ sel, const int32_t *__restrict__ q_pos,
                   const int32_t *__restrict__ seq_len_ptr, int n_q, int n_rows, int row_ctas, int max_blocks,
                   int32_t *__restrict__ sel_ws, int32_t *counts, uint4 *__restrict__ q16,
                   float *__restrict__ unit, int32_t *dev_err) {
    const int l = threadIdx.x & 15;
    if ((int)blockIdx.x >= row_ctas) {
        const int i = ((int)blockIdx.x - row_ctas) * 16 + (threadIdx.x >> 4);
        pdl_wait();   // the selection may come from the kernel before, as the zeroed counts do
        if (i >= n_q) return;
        const int len = __ldg(seq_len_ptr), p = __ldg(q_pos + i);
        const bool ok = p >= 0 && p < len && len <= max_blocks * kBlock;
        if (!ok && l == 0) flag_error(dev_err, UOCR_DEVERR_POS);
        int j = ok ? __ldcg(sel + (size_t)i * kSel + l) : -1;
        if (j > p / kBlock) {
            flag_error(dev_err, UOCR_DEVERR_SEL);
            j = -1;
        }
        if (j < 0) j = -1;
        sel_ws[(size_t)i * kSel + l] = j;
        if (j >= 0) atomicAdd(counts + j, 1);
        return;
    }
    const int row = blockIdx.x * 16 + (threadIdx.x >> 4);
    const bool live = row < n_rows;
    float x[8];
    float amax = 0.f;
    bf16x8_to_f32(live ? __ldg(q + (size_t)row * 16 + l) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float inv;
    const float s = f16_row_scale(amax, inv);
    pdl_wait();   // the workspace may still be read by the call before
    if (!live) return;
    // dims 8 l ..: half l / 8, c = (l % 8) / 2, x % 2 = l % 2
    const int piece = 4 * (2 * (l >> 3) + (l & 1)) + ((l & 7) >> 1);
    q16[(size_t)row * 16 + piece] = make_uint4(pack_f16(x[0] * s, x[1] * s), pack_f16(x[2] * s, x[3] * s),
                                               pack_f16(x[4] * s, x[5] * s), pack_f16(x[6] * s, x[7] * s));
    if (l == 0) unit[row] = inv;
}

__global__ void __launch_bounds__(kBlkWarps * 32, kBlkCtas)
kv8_block_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const uint4 *__restrict__ q16, const float *__restrict__ unit, const float *__restrict__ k_scale,
                 const float *__restrict__ v_scale, const int2 *__restrict__ list, const int4 *__restrict__ items,
                 const int32_t *__restrict__ n_items, int H, int num_pages, float scale_log2,
                 uint4 *__restrict__ part_o, float4 *__restrict__ part_ml, int32_t *dev_err, uint64_t first_wait_ns) {
    extern __shared__ uint8_t raw_smem[];
    __shared__ uint64_t s_bar[kBlkWarps][2];   // K and Q, V of the warp's unit
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint64_t *bar_k = &s_bar[warp][0], *bar_v = &s_bar[warp][1];
    const uint32_t area = ((smem_addr(raw_smem) + 1023u) & ~1023u) + warp * (uint32_t)sizeof(UnitSmem);
    const uint32_t at_k = area + offsetof(UnitSmem, k), at_v = area + offsetof(UnitSmem, v);
    const uint32_t at_q = area + offsetof(UnitSmem, q);
    // this lane's pieces: K piece c of row rho(g) of an 8-row group (piece c + 4 is 64 bytes away by xor,
    // the next group 1024 bytes on); V piece g of row r0 (row r0 ^ 4: by xor); Q piece c of row g
    const int rho = ((g & 1) << 2) | (g >> 1), r0 = c + 4 * (c & 1);
    const uint32_t my_k = at_k + rho * kD + ((c ^ rho) << 4);
    const uint32_t my_v = at_v + r0 * kD + ((g ^ r0) << 4);
    const uint32_t my_q = at_q + g * kQStride + (c << 4);
    if (lane == 0) {
        mbar_init(bar_k, 1);
        mbar_init(bar_v, 1);
        fence_mbar_init();
    }
    __syncwarp();
    uint64_t keep, once;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
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
        if (!page_ok(rec)) return;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_k, kTile8 + rec.w * (kD * 2));
            tma_tile(at_k, &map_k, rec.y * H + h, bar_k, once);
        }
        __syncwarp();
        // row r by lane 4 (r & 7) + r / 8 (it has the entry); rows past the item's end are left as they
        // are: what is computed from them is not stored
        const int row = g + 8 * c;
        if (c < 2 && row < rec.w)
            bulk_row(at_q + row * kQStride, q16 + ((size_t)((c ? eb.x : ea.x) >> 4) * H + h) * 16, kD * 2, bar_k);
    };
    auto issue_v = [&](const int4 &rec, int h) {
        if (page_ok(rec) && lane == 0) {
            mbar_arrive_expect_tx(bar_v, kTile8);
            tma_tile(at_v, &map_v, rec.y * H + h, bar_v, once);
        }
    };
    uint32_t parity = 0;
    // a wait ran out and what follows is left empty; K's copy still on its way: 1 none, 2 the unit's
    // that follows (parity), 3 the unit's own (parity ^ 1)
    int dead = 0;

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
        const bool good = page_ok(rec) && !dead;
        float vs = 0.f, ks = 0.f, ua = 0.f, ub = 0.f;
        if (good) {
            const size_t tile = (size_t)rec.y * H + h;
            ks = __ldg(k_scale + tile);
            vs = __ldg(v_scale + tile);
            ua = __ldcg(unit + row_a);
            ub = __ldcg(unit + row_b);
        } else if (lane == 0 && !dead) {
            flag_error(dev_err, UOCR_DEVERR_PAGE);
        }

        // ---- S: rows g, g + 8; tokens 8 nt + c, 8 nt + 4 + c
        const bool ok_k = __all_sync(0xffffffffu, !good || mbar_wait_timed(bar_k, parity, first_wait_ns, nullptr));
        float s[4][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            uint4 k[4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) k[nt] = ld_smem((my_k ^ (64u * f)) + 1024u * nt);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint4 a = ld_smem(my_q + 64u * (2 * f + y)), b = ld_smem(my_q + 8 * kQStride + 64u * (2 * f + y));
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
        __syncwarp();   // K and Q are read: the next unit's may land
        if (!dead && ok_k) issue_qk(rec1, at1.h, ea1, eb1);

        // ---- causal mask, maxima, weights
        const int t0 = rec.x * kBlock;
        const int far = __reduce_max_sync(0xffffffffu, max(ea.y, eb.y)) - t0 + 1;
        const int near = __reduce_min_sync(0xffffffffu, min(ea.y, eb.y)) - t0 + 1;
        // z = s fa (rows g), s fb: the maximum is taken over s, whose sign the factors then do not change,
        // and a weight is 2^((s - max) fa): 1 at the maximum and at most 1 elsewhere, however large the
        // scores are.  (2^(s fa - ma) with the product kept exact is one instruction less, but its exponent
        // at the maximum is the rounding of ma: from scores of 2^27 on that leaves fp16's range.)
        if ((ks < 0.f) != (scale_log2 < 0.f)) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = -s[nt][e];
        }
        const float fa = fabsf(score_factor(ua, ks, scale_log2)), fb = fabsf(score_factor(ub, ks, scale_log2));
        const bool partly = near < kBlock;   // some query does not see the whole block
        auto hidden = [&](int nt, int e, int pos) { return t0 + 8 * nt + 4 * e + c > pos; };
        if (partly) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (hidden(nt, e, ea.y)) s[nt][e] = -INFINITY;
                    if (hidden(nt, e, eb.y)) s[nt][2 + e] = -INFINITY;
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
        // the states' units are 2^ma, 2^mb (every score NaN or -inf: 2^0, and the sums say which)
        const float sa = ma == -INFINITY ? 0.f : ma, sb = mb == -INFINITY ? 0.f : mb;
        ma = sa * fa;
        mb = sb * fb;
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                p[e] = exp2_approx((s[nt][e] - sa) * fa);
                p[2 + e] = exp2_approx((s[nt][2 + e] - sb) * fb);
            }
            if (partly) {   // (-inf times a scale of 0 is not -inf)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (hidden(nt, e, ea.y)) p[e] = 0.f;
                    if (hidden(nt, e, eb.y)) p[2 + e] = 0.f;
                }
            }
            la += p[0] + p[1];
            lb += p[2] + p[3];
            pa[nt] = pack_f16(p[0], p[1]);
            pb[nt] = pack_f16(p[2], p[3]);
        }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            la += __shfl_xor_sync(0xffffffffu, la, x);
            lb += __shfl_xor_sync(0xffffffffu, lb, x);
        }

        // ---- O = P V8: rows g, g + 8; column n of MMA e is dim 16 n + e
        const bool ok = __all_sync(0xffffffffu, (!good || mbar_wait_timed(bar_v, parity, kWaitLimitNs, nullptr)) && ok_k);
        if (good) parity ^= 1;
        auto v_token = [&](int x) { return 8 * (x >> 1) + (x & 1 ? r0 ^ 4 : r0); };
        auto v_piece = [&](int x) { return ld_smem((x & 1 ? my_v ^ (4u * kD + 64u) : my_v) + 1024u * (x >> 1)); };
        // A token behind a query's position has weight 0, but 0 * NaN is not 0.  Tokens that no query
        // of the item sees may hold anything and are cut off for all of them; where some queries see
        // a token that others do not and its value is NaN, each row gets a product of its own.
        bool apart = false;
        if (near < min(far, kBlock)) {
            uint32_t nan = 0u;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint4 v = v_piece(x);
                if (v_token(x) < far)
#pragma unroll
                    for (int w = 0; w < 4; ++w) nan |= __vcmpeq4(word(v, w) & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
            apart = __any_sync(0xffffffffu, nan != 0u);
        }
        const uint32_t sel_lo = c & 1 ? 0x1504u : 0x5140u, sel_hi = c & 1 ? 0x3726u : 0x7362u;
#pragma unroll 1
        for (int turn = 0; turn < (apart ? kRows : 1); ++turn) {
            int seen = far;
            bool want_a = g < rec.w, want_b = g + 8 < rec.w;
            if (apart) {
                seen = __shfl_sync(0xffffffffu, turn < 8 ? ea.y : eb.y, 4 * (turn & 7)) - t0 + 1;
                want_a = want_a && turn == g;
                want_b = want_b && turn == g + 8;
            }
            // piece 4 w4 + c of a partial holds dims 32 c + 4 w4 .. + 3 and 32 c + 16 + 4 w4 .. + 3: what a
            // lane has at one step, so that a row's four lanes write 64 bytes together
            uint4 *dst_a = part_o + ((size_t)row_a * kSel + (ea.x & 15)) * 16 + c;
            uint4 *dst_b = part_o + ((size_t)row_b * kSel + (eb.x & 15)) * 16 + c;
            uint4 v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = v_piece(x);
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
                    to_f16_here(__byte_perm(t0w, t1w, sel_lo), b0[0], b0[1]);
                    to_f16_here(__byte_perm(t0w, t1w, sel_hi), b0[2], b0[3]);
                    to_f16_here(__byte_perm(t2w, t3w, sel_lo), b1[0], b1[1]);
                    to_f16_here(__byte_perm(t2w, t3w, sel_hi), b1[2], b1[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kk == 0)
                            mma_f16_new(o[e], pa[0], pb[0], pa[1], pb[1], b0[e], b1[e]);
                        else
                            mma_f16(o[e], pa[2], pb[2], pa[3], pb[3], b0[e], b1[e]);
                    }
                }
                if (want_a)
                    st_keep(dst_a + 4 * w4, make_uint4(pack_f16(o[0][0], o[1][0]), pack_f16(o[2][0], o[3][0]),
                                                       pack_f16(o[0][1], o[1][1]), pack_f16(o[2][1], o[3][1])), keep);
                if (want_b)
                    st_keep(dst_b + 4 * w4, make_uint4(pack_f16(o[0][2], o[1][2]), pack_f16(o[2][2], o[3][2]),
                                                       pack_f16(o[0][3], o[1][3]), pack_f16(o[2][3], o[3][3])), keep);
            }
        }
        __syncwarp();   // V is read: the next unit's may land
        if (!ok) {      // a copy did not arrive in time: nothing of this unit and of those after it is kept
            if (lane == 0 && !dead) flag_error(dev_err, UOCR_DEVERR_TIMEOUT);
            if (!dead) dead = !ok_k ? 3 : page_ok(rec1) ? 2 : 1;
        }
        if (!dead) issue_v(rec1, at1.h);

        const bool full = good && ok;   // else (also: a page outside the pool) the states are empty
        if (c == 0) {
            if (g < rec.w)
                part_ml[(size_t)row_a * kSel + (ea.x & 15)] = make_float4(full ? ma : -INFINITY, full ? la : 0.f, vs, 0.f);
            if (g + 8 < rec.w)
                part_ml[(size_t)row_b * kSel + (eb.x & 15)] = make_float4(full ? mb : -INFINITY, full ? lb : 0.f, vs, 0.f);
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
    if (dead) {   // copies still on their way end before the shared memory goes
        if (dead > 1) mbar_drain(bar_k, dead == 2 ? parity : parity ^ 1, dev_err);
        mbar_drain(bar_v, parity ^ 1, dev_err);
    }
}

__global__ void __launch_bounds__(kMrgWarps * 32, 2)
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
        v[s] = ld_l2(part_o + (slot + s) * 16 + k, has);
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
    // piece k = 4 w4 + c of a partial holds dims 32 c + 4 w4 .. + 3 and 32 c + 16 + 4 w4 .. + 3
    uint2 *to = reinterpret_cast<uint2 *>(out + (size_t)ih * 16) + 8 * (k & 3) + (k >> 2);
    to[0] = make_uint2(r[0], r[1]);
    to[4] = make_uint2(r[2], r[3]);
    if (mass_fx && some) {
        atomicAdd(mass_fx + (size_t)h * max_blocks + j, fixed_weight(w / L));
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

namespace {
// A cache of codes as a 3-D tensor (dim, token, page * H + head), read in boxes of one tile.
bool tile8_map(CUtensorMap *map, const void *cache, int num_pages, int H) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)kBlock, (cuuint64_t)num_pages * H};
    const cuuint64_t strides[2] = {(cuuint64_t)kD, (cuuint64_t)kTile8};
    const cuuint32_t box[3] = {(cuuint32_t)kD, (cuuint32_t)kBlock, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(cache), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

size_t prefill_kv8_workspace(int n_q, int H, int max_blocks) { return layout(n_q, H, max_blocks).total; }

namespace {
// Few rows: a query at a time (sparse_attn_kv8_kernel), as long as all its CTAs are resident at once.
// The block by block form has five launches where that has one (three with totals), and reads a
// block once where that reads it once per query.  Measured, blocks / queries (us, both with totals, 10
// heads): over 4000 tokens 1 query 12.5 / 7.4, 16: 14.0 / 10.3, 50: 15.2 / 15.0, 74: 16.1 / 17.2, 100: 16.7 /
// 25.6; over 60000 1: 13.6 / 7.6, 16: 17.8 / 10.8, 50: 25.1 / 16.5, 74: 27.1 / 19.1, 100: 29.4 / 30.1.
bool per_query(const LaunchCtx &c, int n_q, int H) { return (long long)n_q * H <= 5ll * c.num_sms; }
}  // namespace

cudaError_t zero_prefill_kv8(const LaunchCtx &c, void *ws, int n_q, int H, int max_blocks, bool totals,
                             int32_t **sched) {
    const Kv8PrefillWs w = layout(n_q, H, max_blocks);
    char *base = (char *)ws;
    if (sched) *sched = (int32_t *)(base + w.sched_off);
    // what is needed: [counts, list counters], the scoring's counter, [sums]
    const size_t from = !per_query(c, n_q, H) ? 0 : sched ? w.sched_off : w.mass_off;
    const size_t to = totals ? w.zero_bytes : w.mass_off;
    return from < to ? cudaMemsetAsync(base + from, 0, to - from, c.stream) : cudaSuccess;
}

cudaError_t launch_prefill_kv8(const LaunchCtx &c, const void *q, const Kv8Cache &kv, const int32_t *bt,
                               const int32_t *seq_lens, int seq, const int32_t *q_pos, const int32_t *sel, int n_q,
                               int B, int H, int max_blocks, int num_pages, float scale, void *out, float *mass,
                               void *ws, int32_t *dev_err) {
    const int32_t *bt_row = bt + (size_t)seq * max_blocks, *seq_len_ptr = seq_lens + seq;
    float *mass_row = mass ? mass + (size_t)seq * H * max_blocks : nullptr;
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
    auto add_totals = [&]() {
        const int n = H * max_blocks;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)((n + 255) / 256));
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, kv8_totals_kernel, (const unsigned long long *)mass_fx, n, mass_row);
    };
    if (per_query(c, n_q, H)) {
        // (after the selection kernel of a whole step its slots have the layout that it gives them)
        const cudaError_t e = launch_sparse_attn_kv8(c, q, kv, bt, seq_lens, nullptr, q_pos, sel, n_q, B, H, max_blocks,
                                                     num_pages, scale, out, nullptr, c.pdl, dev_err, seq, mass_fx);
        return e != cudaSuccess || !mass_row ? e : add_totals();
    }
    cfg.numAttrs = c.pdl ? 1 : 0;
    const int n_rows = n_q * H, row_ctas = (n_rows + 15) / 16;   // below 2^30 rows
    cfg.gridDim = dim3((unsigned)(row_ctas + (n_q + 15) / 16));
    cfg.blockDim = dim3(256);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_prepare_kernel, (const uint4 *)q, sel, q_pos, seq_len_ptr, n_q, n_rows,
                                       row_ctas, max_blocks, sel_ws, counts, q16, unit, dev_err);
    if (e != cudaSuccess) return e;
    e = launch_prefill_invert(c, counts, bt_row, sel_ws, q_pos, n_q, max_blocks, (int32_t *)(base + w.fill_off), items,
                              n_items, list);
    if (e != cudaSuccess) return e;

    cfg.numAttrs = 1;
    CUtensorMap map_k, map_v;
    if (!tile8_map(&map_k, kv.k, num_pages, H) || !tile8_map(&map_v, kv.v, num_pages, H)) return cudaErrorInvalidValue;
    constexpr int kSmem = kBlkWarps * (int)sizeof(UnitSmem) + 1024;
    e = cudaFuncSetAttribute(kv8_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(kBlkCtas * c.num_sms));
    cfg.blockDim = dim3(kBlkWarps * 32);
    cfg.dynamicSmemBytes = kSmem;
    e = cudaLaunchKernelEx(&cfg, kv8_block_kernel, map_k, map_v, (const uint4 *)q16, (const float *)unit, kv.k_scale,
                           kv.v_scale, (const int2 *)list, (const int4 *)items, (const int32_t *)n_items, H, num_pages,
                           scale * kLog2e, part_o, ml, dev_err, c.first_wait_ns);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;

    cfg.gridDim = dim3((unsigned)((n_rows + 2 * kMrgWarps - 1) / (2 * kMrgWarps)));
    cfg.blockDim = dim3(kMrgWarps * 32);
    e = cudaLaunchKernelEx(&cfg, kv8_merge_kernel, (const int32_t *)sel_ws, (const uint4 *)part_o, (const float4 *)ml,
                           n_rows, H, max_blocks, (uint4 *)out, mass_fx);
    return e != cudaSuccess || !mass_row ? e : add_totals();
}

}  // namespace uocr
