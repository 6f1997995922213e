// The softmax of a tile of 128 query rows x 128 keys between two tensor-core
// products, shared by the prompt kernel and the shared-prefix kernel.
//
// S lies in tensor memory (fp32, 128 columns) and P goes over it (16-bit, 64
// columns), O beside it (fp32).  With the running maximum m and sum l of a
// row, a tile of keys adds
//   p_j = 2^(c s_j - c m),  l += sum_j p_j,  o += sum_j p_j v_j    (c = scale log2 e)
// and where a tile raises the maximum, l and o are first multiplied by
// 2^(c m_old - c m_new).  o only needs m to be near the maximum: it stays
// where it is until a tile exceeds it by 2^8 (p then reaches 256, which costs
// neither 16-bit p nor the fp32 sums any digits), so o is rescaled a few times
// per row and not once per tile.
//
// A warp holds 16 rows, four lanes a row: lane (g, t) = (lane / 4, lane % 4)
// has keys 8 i + 2 t and 8 i + 2 t + 1 of rows g and g + 8.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_plan.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // log2 of how far p may exceed 1 before m moves
// f16 holds 11 digits down to 2^-14 only, so where P is f16 all of p, in the sum l as
// in P, is taken 2^7 times (it reaches 2^15 with the slack): weights keep their digits
// down to 2^-21 of the largest one.  (One token with nearly all of the weight and a
// value near 0 leaves the result to such weights: 2000 of 2^-20.6 were 4% off.)
constexpr float kLift = 7.0f;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two E4M3 codes (low or high half of u) -> two f16 values, exact.
__device__ __forceinline__ uint32_t f16_lo(uint32_t u) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(r)
        : "r"(u));
    return r;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t u) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(u));
    return r;
}

// 2^n, for n beyond fp32's exponents too (as two factors).
__device__ __forceinline__ float scaled(float x, int n) {
    const int h = n / 2;
    return x * __uint_as_float(static_cast<uint32_t>(127 + h) << 23) *
           __uint_as_float(static_cast<uint32_t>(127 + n - h) << 23);
}

// A query row goes to f16 with its largest element in [2^14, 2^15), which is
// exact down to 2^-38 of that element; `top` is the row's largest bf16
// magnitude (bits).  The power of two taken out: 14 - exponent.
__device__ __forceinline__ int query_shift(uint32_t top) {
    return top == 0 ? 0 : 14 - (max(static_cast<int>(top >> 7), 1) - 127);
}

__device__ __forceinline__ uint32_t top_of(const uint4& u, uint32_t top) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    return top;
}

// The running maximum (of s, not of c s) and sum of a lane's two rows; each
// lane sums its own keys, in two parts.
struct SoftmaxRows {
    float m[2] = {-INFINITY, -INFINITY};
    float l[2][2] = {};

    // The whole row's sum.
    __device__ float sum(int e) const {
        float v = l[e][0] + l[e][1];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    }
};

__device__ __forceinline__ void load_scores(uint32_t tS, uint32_t (&s)[4][16]) {
#pragma unroll
    for (int b = 0; b < 4; ++b) tmem_ld_16x256b_x4(tS + 32 * b, s[b]);
    tmem_ld_wait();
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(s[b][i]));  // (no use before the wait)
}

// Hides keys 2 t + ... beyond `seen` (counted from key 2 t of the tile) from row e.
__device__ __forceinline__ void hide_after(uint32_t (&s)[4][16], int e, int seen) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (32 * b + 8 * (i >> 1) + (i & 1) > seen)
                s[b][4 * (i >> 1) + 2 * e + (i & 1)] = 0xFF800000u;  // -inf
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// P of 64 keys (half b of the tile) from their scores, and its sums.
template <bool kBf16>
__device__ __forceinline__ void weights_of(const uint32_t (&s)[4][16], int b, const float (&c)[2],
                                           const float (&base)[2], uint32_t (&p)[16], float (&sum)[2][2]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        // keys 64 b + 8 (i / 2) + 2 t, + 1 of row i & 1
        const int e = i & 1;
        const uint32_t* from = &s[2 * b + (i >> 3)][4 * (i >> 1 & 3) + 2 * e];
        float y0 = base[e], y1 = base[e];
        fma2(y0, y1, __uint_as_float(from[0]), __uint_as_float(from[1]), c[e], c[e]);
        y0 = ex2(y0);
        y1 = ex2(y1);
        add2(sum[e][0], sum[e][1], y0, y1);
        p[i] = kBf16 ? pack_bf16(y0, y1) : pack_f16(y0, y1);
    }
}

// P of the tile from its scores; `started`: O holds earlier tiles.  c: scale
// log2(e) of each row; real: rows that count.  `half` is called when the P of
// 64 keys is in tensor memory.
//
// kAhead: the maximum as a rule stays where it is, so the first half's P is
// taken with the old one while the tile's maximum is still being found (300
// clocks of comparisons and shuffles, which the tensor core would wait for),
// and taken again if that turns out too small.  It costs some 20 registers.
template <bool kBf16, int DP, bool kAhead, typename Half>
__device__ __forceinline__ void softmax_tile(uint32_t (&s)[4][16], uint32_t tS, uint32_t tO,
                                             SoftmaxRows& rows, const float (&c)[2],
                                             const bool (&real)[2], bool started, Half half) {
    constexpr float lift = kBf16 ? 0.0f : kLift;
    float base[2] = {rows.m[0] == -INFINITY ? 0.0f : lift - rows.m[0] * c[0],
                     rows.m[1] == -INFINITY ? 0.0f : lift - rows.m[1] * c[1]};
    uint32_t p[16];
    float sum[2][2] = {};
    if (kAhead) weights_of<kBf16>(s, 0, c, base, p, sum);
    float top[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float part[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            part[b] = fmaxf(__uint_as_float(s[b][2 * e]), __uint_as_float(s[b][2 * e + 1]));
#pragma unroll
            for (int i = 2; i < 8; i += 2)
                part[b] = max3(part[b], __uint_as_float(s[b][4 * (i >> 1) + 2 * e]),
                               __uint_as_float(s[b][4 * (i >> 1) + 2 * e + 1]));
        }
        top[e] = fmaxf(max3(part[0], part[1], part[2]), part[3]);
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xFFFFFFFFu, top[0], d));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xFFFFFFFFu, top[1], d));
    }
    bool raise[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)  // (m = -inf: the first keys that are seen set it)
        raise[e] = real[e] && (top[e] - rows.m[e]) * c[e] > kSlack;
    if (__any_sync(0xFFFFFFFFu, raise[0] || raise[1])) {
        // (row by row, so that no row's digits depend on its neighbours)
        float keep[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            keep[e] = !raise[e] ? 1.0f : rows.m[e] == -INFINITY ? 0.0f : ex2((rows.m[e] - top[e]) * c[e]);
            rows.m[e] = raise[e] ? top[e] : rows.m[e];
            rows.l[e][0] *= keep[e];
            rows.l[e][1] *= keep[e];
            base[e] = rows.m[e] == -INFINITY ? 0.0f : lift - rows.m[e] * c[e];
            sum[e][0] = sum[e][1] = 0.0f;
        }
        if (started) {
            // S of this tile came after P V of the one before: O is at rest
#pragma unroll 1
            for (int b = 0; b < DP / 32; ++b) {
                uint32_t o[16];
                tmem_ld_16x256b_x4(tO + 32 * b, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+r"(o[i]));
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * keep[i >> 1 & 1]);
                }
                tmem_st_16x256b_x4(tO + 32 * b, o);
            }
        }
        if (kAhead) weights_of<kBf16>(s, 0, c, base, p, sum);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (b == 1 || !kAhead) weights_of<kBf16>(s, b, c, base, p, sum);
        tmem_st_16x128b_x8(tS + 32 * b, p);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        half(b);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        rows.l[e][0] += sum[e][0];
        rows.l[e][1] += sum[e][1];
    }
}

}  // namespace fp8k
