// The end of a block and the start of the next, in one pass over the tokens:
//   b  = sum_j w[t, j] y[row[t, j]]  or  y[t]
//   b  = b / sqrt(mean b^2 + eps) gamma_post        (with gamma_post)
//   b  = b gate                                     (with a gate)
//   h' = residual_scale h + branch_scale b          -> bf16
//   z  = h' / sqrt(mean h'^2 + eps) gamma           -> bf16
//   s  = amax |z| / 448, codes = E4M3(z / s)
//
// A group of G threads owns a token and keeps its row in registers in fp32,
// 8 elements (a 16-byte load) a chunk, so that every tensor is read once and
// each result is rounded once.  Up to three reductions over the row follow one
// another (sum of squares of b, of h', maximum of z); several CTAs an SM hide
// them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

constexpr int kBlock = 256;

template <int G, bool kMax>
__device__ __forceinline__ float over_row(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    if constexpr (G > 32) {
        constexpr int WPG = G / 32;
        const int warp = threadIdx.x >> 5;
        if (lane_id() == 0) red[warp] = v;
        __syncthreads();
        const int first = (warp / WPG) * WPG;
        v = red[first];
#pragma unroll
        for (int w = 1; w < WPG; ++w) v = kMax ? fmaxf(v, red[first + w]) : v + red[first + w];
        __syncthreads();
    }
    return v;
}

// (plain loads: what earlier kernels write may not come through the read-only path)
__device__ __forceinline__ uint4 load(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void widen(const uint4& u, float (&v)[8]) {
    v[0] = bf16lo(u.x), v[1] = bf16hi(u.x), v[2] = bf16lo(u.y), v[3] = bf16hi(u.y);
    v[4] = bf16lo(u.z), v[5] = bf16hi(u.z), v[6] = bf16lo(u.w), v[7] = bf16hi(u.w);
}

__device__ __forceinline__ uint32_t pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
    return make_uint4(pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7]));
}

__device__ __forceinline__ float quotient(float x, const Divisor& d) {
    return d.ieee ? __fdiv_rn(x, d.s) : div_rn(x, d);
}

template <int G, int VPT>
__global__ void __launch_bounds__(G > kBlock ? G : kBlock) residual_norm(const ResidualNormArgs a) {
    constexpr int B = G > kBlock ? G : kBlock;
    constexpr int ROWS = B / G;
    __shared__ float red[B / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / G;
    const int i0 = threadIdx.x % G;
    const bool live = t < a.T;
    const int C = static_cast<int>(a.K >> 3);
    const float K = static_cast<float>(a.K);

    float b[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
    if (live) {
        for (int j = 0; j < max(a.k, 1); ++j) {
            const int64_t row = a.k > 0 ? a.token_row[t * a.k + j] : t;
            if (row < 0 || row >= a.R) continue;
            const float w = a.k > 0 && a.weights ? a.weights[t * a.k + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = i0 + i * G;
                if (c < C) {
                    float v[8];
                    widen(load(a.y + row * a.ldy + 8 * c), v);
#pragma unroll
                    for (int l = 0; l < 8; ++l) b[i][l] = fmaf(w, v[l], b[i][l]);
                }
            }
        }
    }
    if (a.gamma_post) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(b[i][j], b[i][j], ss);
        ss = over_row<G, false>(ss, red);
        const float inv = 1.0f / sqrtf(ss / K + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = i0 + i * G;
            if (live && c < C) {
                float g[8];
                widen(load(a.gamma_post + 8 * c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[i][j] = b[i][j] * inv * g[j];
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = i0 + i * G;
        if (live && c < C) {
            if (a.gate) {
                float g[8];
                widen(load(a.gate + t * a.ldg + 8 * c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[i][j] *= g[j];
            }
            float h[8];
            widen(load(a.h + t * a.ldh + 8 * c), h);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                b[i][j] = fmaf(a.residual_scale, h[j], a.branch_scale * b[i][j]);
                ss = fmaf(b[i][j], b[i][j], ss);
            }
            *reinterpret_cast<uint4*>(a.h_out + t * a.ldho + 8 * c) = narrow(b[i]);
        }
    }
    if (!a.z && !a.q) return;
    ss = over_row<G, false>(ss, red);
    const float inv = 1.0f / sqrtf(ss / K + a.eps);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = i0 + i * G;
        if (live && c < C) {
            float g[8];
            widen(load(a.gamma + 8 * c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                b[i][j] = b[i][j] * inv * g[j];
                m = fmaxf(m, fabsf(b[i][j]));
            }
            if (a.z) *reinterpret_cast<uint4*>(a.z + t * a.K + 8 * c) = narrow(b[i]);
        }
    }
    if (!a.q) return;
    m = over_row<G, true>(m, red);
    if (!live) return;
    const float sc = scale_of(m);
    const Divisor d = divisor_of(sc);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = i0 + i * G;
        if (c < C) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = cvt_e4m3x2(quotient(b[i][2 * j], d), quotient(b[i][2 * j + 1], d));
            *reinterpret_cast<uint2*>(a.q + t * a.ldq + 8 * c) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
    }
    if (i0 == 0) a.s[t] = sc;
}

template <int G, int VPT>
cudaError_t launch(const ResidualNormArgs& a, cudaStream_t st) {
    constexpr int B = G > kBlock ? G : kBlock;
    constexpr int ROWS = B / G;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + ROWS - 1) / ROWS));
    cfg.blockDim = dim3(B);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, residual_norm<G, VPT>, a);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, cudaStream_t st) {
    const int64_t C = a.K / 8;
    if (C <= 32) return launch<32, 1>(a, st);
    if (C <= 64) return launch<64, 1>(a, st);
    if (C <= 128) return launch<128, 1>(a, st);
    if (C <= 256) return launch<256, 1>(a, st);
    if (C <= 512) return launch<256, 2>(a, st);
    if (C <= 1024) return launch<512, 2>(a, st);
    if (C <= 2048) return launch<1024, 2>(a, st);
    return launch<1024, 4>(a, st);
}

}  // namespace fp8k
