// kv8.cuh -- warp-level tile products over a key / value cache held in 8 bits (e4m3).
//
// Cache layout: codes [P][H][32][128] of one byte (a (page, head) tile is 4 KiB, contiguous) and
// one fp32 scale per (page, head) for K and one for V: value = code * scale.  The codes go to the
// tensor cores as they are (mma.sync m16n8k32, e4m3 in, fp32 accumulate); the other operand, a
// query or the softmax weights, is written as a sum of a few e4m3 numbers times powers of 2^-5,
//   x = c0 + 2^-5 c1 + 2^-10 c2,  c0 = e4m3(x), c1 = e4m3(2^5 (x - c0)), ...
// each of which removes at least 5 bits of what is left (x is first scaled to below 2^8), and
// each of which takes one of the 8 columns of B: a decode step has one query row per (sequence,
// head), so the columns cost nothing.  Scales are applied to the fp32 results.
//   - three terms hold a bf16 query to 2^-27 of its row's largest element (a number's 8 bits are
//     exact after two, wherever it is not 2^-14 below the largest);
//   - three terms hold a weight in [0, 1] to 2^-13 of itself;
//   - the products' sums were checked against 64 bits: within 2^-22 of the sum of magnitudes over
//     128 terms (random codes, chained accumulation), as fp32 FMAs would be.
// Measured on a B200 (instructions a clock and SM): this MMA 0.94, m16n8k16 in fp16 0.50, a byte
// permute 2.0, e4m3x2 -> f16x2 1.9; turning codes into fp16 first costs the tile 128 conversions a
// lane and twice the MMAs at half their rate.
//
// Fragments.  The contraction index of an MMA may be permuted as long as both operands agree, so
// lane (g, c) = (lane / 4, lane % 4) takes its operand elements as whole 16-byte pieces of a row,
// straight from global memory into registers (no staging, no shuffles, full 32-byte sectors):
//   K, rows g + 8 i (i = 0..3): pieces c and c + 4 of the row (dims 16 c .. + 15 and 64 + 16 c .. + 15);
//      a register holds 4 dims, two make one 32-dim MMA step of the row;
//   V: piece g (dims 16 g .. 16 g + 15) of the 8 tokens 4 x + c; a 4 x 4 byte transpose (8 permutes)
//      turns four tokens' words into the registers of four dims, four tokens each.
// The scores of tokens g + 8 i come out in quad g, and one register of B holds four tokens of one
// column: a quad's four weights, packed, are what lane c = g % 4 of a column needs.
// These are the warp-level MMAs: a decode step has one query row per (sequence, head), and an item
// of a prefill chunk at most 16, far below the 64-row tile of tcgen05.
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

// d += A (16 x 32, row) * B (32 x 8, col); e4m3 operands, fp32 accumulators.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four numbers (|x| <= 448, or NaN) to packed e4m3 codes, and what is left of them times 32.
__device__ __forceinline__ uint32_t e4m3_term(float (&x)[4]) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
    const uint32_t l = e4m3x2_to_f16x2(lo), h = e4m3x2_to_f16x2(hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&l));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    x[0] = (x[0] - a.x) * 32.f;
    x[1] = (x[1] - a.y) * 32.f;
    x[2] = (x[2] - b.x) * 32.f;
    x[3] = (x[3] - b.y) * 32.f;
    return (uint32_t)lo | (uint32_t)hi << 16;
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

// The power of two that brings a row with largest magnitude amax into [2^kTop, 2^(kTop + 1)), and
// its inverse.
template <int kTop>
__device__ __forceinline__ float row_scale(float amax, float &inverse) {
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;       // amax >= 0; 128 for inf / NaN
    const int k = min(kTop - e, 126);                             // at least kTop - 128
    inverse = __uint_as_float((uint32_t)(127 - k) << 23);
    return __uint_as_float((uint32_t)(127 + k) << 23);
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

// One decode query as the B operand of S^T = K q: columns 0..2 hold its terms, the rest zeros.
struct __align__(16) Query8Smem {
    uint32_t t[4][kD / 4];   // terms 0..2, then zeros
};
struct Query8 {
    uint4 w[2];      // dims 16 c .. + 15 and 64 + 16 c .. + 15 of term g
    float unit;      // the products are in units of this
};
// By a whole warp, through an area of its own; raw: the lane's dims 4 lane .. 4 lane + 3.
__device__ __forceinline__ Query8 split_query8(Query8Smem &sm, uint2 raw, int lane) {
    float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u), __uint_as_float(raw.y << 16),
                  __uint_as_float(raw.y & 0xffff0000u)};
    const float amax = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    Query8 q;
    const float s = row_scale<7>(amax, q.unit);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= s;
    // an infinity saturates in the first term and leaves one to the next: make it NaN there
    bool fine = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) fine = fine && fabsf(x[e]) <= 448.f;
    const uint32_t first = e4m3_term(x);
    sm.t[0][lane] = fine ? first : 0x7f7f7f7fu;
    sm.t[1][lane] = e4m3_term(x);
    sm.t[2][lane] = e4m3_term(x);
    sm.t[3][lane] = 0u;
    __syncwarp();
    const uint4 *src = reinterpret_cast<const uint4 *>(sm.t[min(lane >> 2, 3)]);
    q.w[0] = src[lane & 3];
    q.w[1] = src[4 + (lane & 3)];
    return q;
}

// What a lane's two accumulator columns count for: columns 0, 1, 2 in units of 1, 2^-5, 2^-10.
__device__ __forceinline__ float2 term_units(int lane) {
    const int c = lane & 3;
    return make_float2(c == 0 ? 1.f : c == 1 ? 1.f / 1024.f : 0.f, c == 0 ? 1.f / 32.f : 0.f);
}

// Scores of a K tile, in units of q.unit * scale: every lane of quad g gets those of tokens g, 8 + g,
// 16 + g, 24 + g.
__device__ __forceinline__ void scores8(float (&z)[4], const uint4 (&k)[8], const Query8 &q, int lane) {
    float d[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) d[m][0] = d[m][1] = d[m][2] = d[m][3] = 0.f;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint4 &a = k[4 * m + f], &b = k[4 * m + 2 + f];
            mma_e4m3(d[m], a.x, b.x, a.y, b.y, q.w[f].x, q.w[f].y);
            mma_e4m3(d[m], a.z, b.z, a.w, b.w, q.w[f].z, q.w[f].w);
        }
    const float2 u = term_units(lane);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            // lanes c >= 2 hold columns of zeros
            float t = (lane & 2) ? 0.f : fmaf(d[m][2 * y], u.x, d[m][2 * y + 1] * u.y);
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            z[2 * m + y] = t + __shfl_xor_sync(0xffffffffu, t, 2);
        }
}

// Four words (tokens), bytes = dims, to four words (dims), bytes = tokens.
__device__ __forceinline__ void transpose4(uint32_t (&r)[4], uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
    const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w2, w3, 0x5140);
    const uint32_t c = __byte_perm(w0, w1, 0x7362), d = __byte_perm(w2, w3, 0x7362);
    r[0] = __byte_perm(a, b, 0x5410);
    r[1] = __byte_perm(a, b, 0x7632);
    r[2] = __byte_perm(c, d, 0x5410);
    r[3] = __byte_perm(c, d, 0x7632);
}

// acc[e] += s * sum_t p_t v[t][16 g + e], for the weights p of scores8's tokens; the sum over the
// lanes c = 0, 1 of a quad is the result.
__device__ __forceinline__ void weighted_sum8(float (&acc)[16], const float (&p)[4], const uint4 (&v)[8], float s,
                                              int lane) {
    const int g = lane >> 2, c = lane & 3;
    float x[4] = {p[0] * 256.f, p[1] * 256.f, p[2] * 256.f, p[3] * 256.f};
    const uint32_t t0 = e4m3_term(x), t1 = e4m3_term(x), t2 = e4m3_term(x);
    const uint32_t mine = c == 0 ? t0 : c == 1 ? t1 : c == 2 ? t2 : 0u;
    // column g: term g of quads c (tokens c + 8 i) and c + 4
    uint32_t b0 = __shfl_sync(0xffffffffu, mine, 4 * c + (g & 3));
    uint32_t b1 = __shfl_sync(0xffffffffu, mine, 4 * c + (g & 3) + 16);
    if (g >= 4) b0 = b1 = 0u;
    const float2 u = term_units(lane);
    const float s0 = s * (u.x * (1.f / 256.f)), s1 = s * (u.y * (1.f / 256.f));
#pragma unroll
    for (int w = 0; w < 2; ++w) {   // dims 4 w .. + 3 (rows g) and 8 + 4 w .. + 3 (rows g + 8)
        uint32_t a0[4], a1[4], a2[4], a3[4];
        transpose4(a0, word(v[0], w), word(v[2], w), word(v[4], w), word(v[6], w));
        transpose4(a1, word(v[0], w + 2), word(v[2], w + 2), word(v[4], w + 2), word(v[6], w + 2));
        transpose4(a2, word(v[1], w), word(v[3], w), word(v[5], w), word(v[7], w));
        transpose4(a3, word(v[1], w + 2), word(v[3], w + 2), word(v[5], w + 2), word(v[7], w + 2));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_e4m3(d, a0[e], a1[e], a2[e], a3[e], b0, b1);
            acc[4 * w + e] = fmaf(d[0], s0, fmaf(d[1], s1, acc[4 * w + e]));
            acc[8 + 4 * w + e] = fmaf(d[2], s0, fmaf(d[3], s1, acc[8 + 4 * w + e]));
        }
    }
}

// The weight a block received, as it is added to the running totals: a weight that is not finite
// (a query with infinities or NaN) adds nothing, so that one bad query does not spoil them.
__device__ __forceinline__ float finite_weight(float w) { return w >= 0.f && w <= 3.4e38f ? w : 0.f; }

}  // namespace uocr
