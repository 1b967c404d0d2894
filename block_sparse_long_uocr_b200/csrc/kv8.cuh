// kv8.cuh -- warp-level tile products over a key / value cache held in 8 bits (e4m3).
//
// Cache layout: codes [P][H][32][128] of one byte (a (page, head) tile is 4 KiB, contiguous) and
// one fp32 scale per (page, head) for K and one for V: value = code * scale.  An e4m3 code is an
// fp16 number exactly (4 significant bits, 2^-9 .. 448), so the tile products run on the fp16
// tensor cores with fp32 accumulation and the scale is applied to their fp32 results: neither K
// nor V is rounded again.  A query row is scaled by a power of two to fp16's range (exact, below);
// a softmax weight, at most 1 and relative to its block's largest, is the sum of two fp16 numbers in
// two columns of B, which a single query leaves free: 22 bits of it are kept, down to 2^-25.
//
// The codes cannot go to the tensor cores as they are: mma.sync m16n8k32 on e4m3 operands runs on a
// B200 as two fp16 MMAs and some 17 further instructions (counted: 23.6 issued per MMA with its
// operand loads against 6.6 for the fp16 one), which converts every operand at every use.  Converted
// once, a tile costs a lane 128 conversions (two codes each, 1.9 warp instructions a clock and SM)
// and 32 MMAs (0.5 a clock).
//
// Fragments.  The contraction index of an MMA may be permuted as long as both operands agree, so
// lane (g, c) = (lane / 4, lane % 4) takes its operand elements as whole 16-byte pieces of a row,
// straight from global memory into registers (no staging, no shuffles, full 32-byte sectors):
//   K, rows g + 8 i (i = 0..3): pieces c and c + 4 of the row (dims 16 c .. + 15 and 64 + 16 c .. + 15);
//      word w of piece f holds the 4 dims of one 16-dim MMA step (f, w), two per operand register;
//   V: piece g (dims 16 g .. 16 g + 15) of 4 tokens per 16-token MMA step; a byte permute pairs two
//      tokens' codes of one dim, which is what one operand register holds.
// These are the warp-level MMAs (m16n8k16): a decode step has one query row per (sequence, head),
// and an item of a prefill chunk at most 16, far below the 64-row tile of tcgen05; the products
// are a small part of the time, the point is to take the dot products and their reductions off the
// FMA pipes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace uocr {

constexpr int kTile8 = kBlock * kD;        // bytes of one (page, head) tile of codes
constexpr int kTile8U4 = kTile8 / 16;      // 16-byte pieces of a tile
constexpr int kRowU4 = kD / 16;            // 16-byte pieces of a token's row

// Two e4m3 codes (low, high byte) to two fp16 numbers: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
    return d;
}
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t &lo, uint32_t &hi) {
    lo = e4m3x2_to_f16x2((uint16_t)(v & 0xffffu));
    hi = e4m3x2_to_f16x2((uint16_t)(v >> 16));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// d += A (16 x 16, row) * B (16 x 8, col); fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same into fresh accumulators.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The power of two that brings a row with largest magnitude amax into [2^14, 2^15), and its
// inverse.  A bf16 query times it is an fp16 number exactly down to 2^-28 of the row's largest
// element (below that fp16's subnormals round it, by less than 2^-39 of the largest).
__device__ __forceinline__ float f16_row_scale(float amax, float &inverse) {
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;       // amax >= 0; 128 for inf / NaN
    const int k = min(14 - e, 126);                               // -114 .. 126
    inverse = __uint_as_float((uint32_t)(127 - k) << 23);
    return __uint_as_float((uint32_t)(127 + k) << 23);
}

// What the products of a row in units of `unit` and of a block with scale ks are multiplied by to
// give scores: unit * ks * scale.  unit and ks meet first (unit is as small as the row is large);
// a factor past fp32's range stays finite, so that a product of 0 is a score of 0.  A ks that is not
// finite gives NaN, in every form of the attention.
__device__ __forceinline__ float score_factor(float unit, float ks, float scale) {
    constexpr float kMax = 3.4028235e38f;
    const float f = unit * ks * scale;
    if (fabsf(f) <= kMax) return f;
    const float a = fminf(fmaxf(unit * ks, -kMax), kMax);
    return fminf(fmaxf(a * scale, -kMax), kMax) + (ks - ks);
}

// 2^x to 2 units; 0 below 2^-126.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Word w (0..3) of a 16-byte piece.
__device__ __forceinline__ uint32_t word(const uint4 &v, int w) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; }

// The lane's 8 pieces of a K tile: k[2 i + f] = piece c + 4 f of row g + 8 i.
__device__ __forceinline__ void load_k8(uint4 (&k)[8], const uint4 *__restrict__ tile, int lane) {
    const uint4 *src = tile + (lane >> 2) * kRowU4 + (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int f = 0; f < 2; ++f) k[2 * i + f] = ld_stream(src + i * 8 * kRowU4 + 4 * f);
}

// The lane's 8 pieces of a V tile: v[x] = piece g of token 4 x + c.
__device__ __forceinline__ void load_v8(uint4 (&v)[8], const uint4 *__restrict__ tile, int lane) {
    const uint4 *src = tile + (lane & 3) * kRowU4 + (lane >> 2);
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = ld_stream(src + x * 4 * kRowU4);
}

// Tokens at and past `visible` of a V tile loaded by load_v8 become zeros: rows behind a
// sequence's end may hold anything, the code of NaN among it, and 0 * NaN is not 0.
__device__ __forceinline__ void mask_v8(uint4 (&v)[8], int visible, int lane) {
#pragma unroll
    for (int x = 0; x < 8; ++x)
        if (4 * x + (lane & 3) >= visible) v[x] = make_uint4(0u, 0u, 0u, 0u);
}

// One decode query as the B operand of S^T = K q: column 0 holds the query, the rest zeros.  Its 16
// registers a lane are read from shared memory at each tile (four 16-byte loads): lane c of the
// first quad reads its dims, every other lane zeros.
struct __align__(16) Query8Smem {
    uint2 x[kD / 4];     // fp16, dims 4 i .. 4 i + 3
    uint2 zero[kD / 4];
};
struct Query8 {
    const uint4 *f;      // pieces 0, 1: dims 16 c .. + 15; pieces 8, 9: dims 64 + 16 c .. + 15
    float unit;          // the products are in units of this
};
// By a whole warp, through an area of its own; raw: the lane's dims 4 lane .. 4 lane + 3.
__device__ __forceinline__ Query8 split_query8(Query8Smem &sm, uint2 raw, int lane) {
    const float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u), __uint_as_float(raw.y << 16),
                        __uint_as_float(raw.y & 0xffff0000u)};
    const float amax = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    Query8 q;
    const float s = f16_row_scale(amax, q.unit);
    sm.x[lane] = make_uint2(pack_f16(x[0] * s, x[1] * s), pack_f16(x[2] * s, x[3] * s));
    sm.zero[lane] = make_uint2(0u, 0u);
    __syncwarp();
    q.f = reinterpret_cast<const uint4 *>(lane < 4 ? sm.x : sm.zero) + 2 * (lane & 3);
    return q;
}

// Scores of a K tile, in units of score_factor(q.unit, ..): every lane of quad g gets those of tokens g, 8 + g,
// 16 + g, 24 + g.
__device__ __forceinline__ void scores8(float (&z)[4], const uint4 (&k)[8], const Query8 &q, int lane) {
    float d[2][4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const uint4 b = q.f[8 * (x >> 1) + (x & 1)];   // MMA steps (x / 2, 2 (x % 2)) and the next
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16(word(k[4 * m + (x >> 1)], 2 * (x & 1) + y), a0, a2);
                e4m3x4_to_f16(word(k[4 * m + 2 + (x >> 1)], 2 * (x & 1) + y), a1, a3);
                if (x == 0 && y == 0)
                    mma_f16_new(d[m], a0, a1, a2, a3, b.x, b.y);
                else
                    mma_f16(d[m], a0, a1, a2, a3, y ? b.z : b.x, y ? b.w : b.y);
            }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        // column 0 sits in the lanes with c = 0
        z[2 * m] = __shfl_sync(0xffffffffu, d[m][0], lane & 28);
        z[2 * m + 1] = __shfl_sync(0xffffffffu, d[m][2], lane & 28);
    }
}

// acc[e] += s * sum_t p_t v[t][16 g + e] in the lanes with c = 0, for the weights p of scores8's
// tokens.
__device__ __forceinline__ void weighted_sum8(float (&acc)[16], const float (&p)[4], const uint4 (&v)[8], float s,
                                              int lane) {
    const int g = lane >> 2, c = lane & 3;
    uint32_t x01, x23;
    {
        const __half2 h01 = __floats2half2_rn(p[0], p[1]), h23 = __floats2half2_rn(p[2], p[3]);
        const uint32_t l01 = pack_f16(p[0] - __low2float(h01), p[1] - __high2float(h01));
        const uint32_t l23 = pack_f16(p[2] - __low2float(h23), p[3] - __high2float(h23));
        x01 = c & 1 ? l01 : *reinterpret_cast<const uint32_t *>(&h01);
        x23 = c & 1 ? l23 : *reinterpret_cast<const uint32_t *>(&h23);
    }
    const int src = 4 * c + (g & 1);
    uint32_t b[2][2];
    b[0][0] = __shfl_sync(0xffffffffu, x01, src);         // tokens c, c + 8
    b[0][1] = __shfl_sync(0xffffffffu, x01, src + 16);    // tokens c + 4, c + 12
    b[1][0] = __shfl_sync(0xffffffffu, x23, src);         // the same + 16
    b[1][1] = __shfl_sync(0xffffffffu, x23, src + 16);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (g >= 2) b[k][0] = b[k][1] = 0u;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // dims 4 w + 2 half, + 1 (rows g) and + 8 (rows g + 8)
            float d0[4], d1[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t sel = half ? 0x7362u : 0x5140u;
                uint32_t a0[2], a1[2], a2[2], a3[2];
                e4m3x4_to_f16(__byte_perm(word(v[4 * k], w), word(v[4 * k + 2], w), sel), a0[0], a0[1]);
                e4m3x4_to_f16(__byte_perm(word(v[4 * k], w + 2), word(v[4 * k + 2], w + 2), sel), a1[0], a1[1]);
                e4m3x4_to_f16(__byte_perm(word(v[4 * k + 1], w), word(v[4 * k + 3], w), sel), a2[0], a2[1]);
                e4m3x4_to_f16(__byte_perm(word(v[4 * k + 1], w + 2), word(v[4 * k + 3], w + 2), sel), a3[0], a3[1]);
                if (k == 0) {
                    mma_f16_new(d0, a0[0], a1[0], a2[0], a3[0], b[0][0], b[0][1]);
                    mma_f16_new(d1, a0[1], a1[1], a2[1], a3[1], b[0][0], b[0][1]);
                } else {
                    mma_f16(d0, a0[0], a1[0], a2[0], a3[0], b[1][0], b[1][1]);
                    mma_f16(d1, a0[1], a1[1], a2[1], a3[1], b[1][0], b[1][1]);
                }
            }
            const int e = 4 * w + 2 * half;
            acc[e] = fmaf(s, d0[0] + d0[1], acc[e]);
            acc[e + 8] = fmaf(s, d0[2] + d0[3], acc[e + 8]);
            acc[e + 1] = fmaf(s, d1[0] + d1[1], acc[e + 1]);
            acc[e + 9] = fmaf(s, d1[2] + d1[3], acc[e + 9]);
        }
    }
}

// The weight a block received, as it is added to the running totals: a weight that is not finite
// (a query with infinities or NaN) adds nothing, so that one bad query does not spoil them.
__device__ __forceinline__ float finite_weight(float w) { return w >= 0.f && w <= 3.4e38f ? w : 0.f; }
// The same as a multiple of 2^-40, for sums whose order is not fixed.
constexpr float kMassUnit = 1.f / (1ll << 40);
__device__ __forceinline__ unsigned long long fixed_weight(float w) {
    return __float2ull_rn(finite_weight(w) / kMassUnit);
}

}  // namespace uocr
