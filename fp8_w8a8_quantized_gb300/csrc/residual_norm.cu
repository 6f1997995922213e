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
// each result is rounded once.  Everything that a token needs is asked for at its
// start or ahead of the reduction before it is used: up to three reductions over
// the row follow one another (sum of squares of b, of h', maximum of z), and
// several CTAs an SM hide them.  Bound by DRAM, with the instructions close
// behind: arithmetic is on pairs (f32x2), and z is kept negated, which is what the
// quantizer's division wants (quant_math.cuh).  8192 tokens of 4096: 49 us, 6.2 TB/s
// (91% of a copy) with y as it is, 55 us with a norm and a gate, 63 us with two rows
// of y by weight, whose places each token has to read first.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

// Threads of a CTA: a token's, so that no token waits at another's barriers; warps that have a
// token to themselves come in eights.
template <int G>
constexpr int kBlockOf = G > 32 ? G : 256;

// Threads an SM: with four chunks a thread half as many, with twice the registers.
template <int VPT>
constexpr int kResident = VPT > 2 ? 512 : 1024;

// Sum or maximum over a token's threads; `red` holds a float a warp and is used once.
template <int G, bool kMax>
__device__ __forceinline__ float over_row(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    if constexpr (G > 32) {
        constexpr int WPG = G / 32;
        if (lane_id() == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < WPG; ++w) v = kMax ? fmaxf(v, red[w]) : v + red[w];
    }
    return v;
}

// (plain loads: what earlier kernels write may not come through the read-only path)
__device__ __forceinline__ uint4 load(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// Two fp32 values -> a bf16 pair, `lo` in the low half.
__device__ __forceinline__ uint32_t pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8], uint32_t flip = 0) {
    return make_uint4(pair(v[0], v[1]) ^ flip, pair(v[2], v[3]) ^ flip, pair(v[4], v[5]) ^ flip, pair(v[6], v[7]) ^ flip);
}

// v += s * u, v *= u, v *= s, and the sum of squares of v into (s0, s1).
__device__ __forceinline__ void add_scaled(float (&v)[8], float s, const uint4& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) fma2(v[2 * i], v[2 * i + 1], bf16lo(word(u, i)), bf16hi(word(u, i)), s, s);
}
__device__ __forceinline__ void times(float (&v)[8], const uint4& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mul2(v[2 * i], v[2 * i + 1], v[2 * i], v[2 * i + 1], bf16lo(word(u, i)), bf16hi(word(u, i)));
}
__device__ __forceinline__ void times(float (&v)[8], float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mul2(v[2 * i], v[2 * i + 1], v[2 * i], v[2 * i + 1], s, s);
}
__device__ __forceinline__ void squares(const float (&v)[8], float& s0, float& s1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) fma2(s0, s1, v[2 * i], v[2 * i + 1], v[2 * i], v[2 * i + 1]);
}

// Codes of -v / s: the steps of quant2 (quant_math.cuh) on fp32 values, which |v| <= 448 s bounds.
__device__ __forceinline__ uint2 codes_of_negated(const float (&v)[8], const Divisor& d) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float z0 = v[2 * i], z1 = v[2 * i + 1];
        if (d.ieee) {
            c[i] = cvt_e4m3x2(__fdiv_rn(-z0, d.s), __fdiv_rn(-z1, d.s));
            continue;
        }
        float q0, q1;
        mul2(q0, q1, z0, z1, d.nr, d.nr);
        float e0 = z0, e1 = z1;
        fma2(e0, e1, q0, q1, d.s, d.s);
        float y0 = q0, y1 = q1;
        fma2(y0, y1, e0, e1, d.nr, d.nr);
        c[i] = cvt_e4m3x2(y0, y1);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// kTop: the branch is rows of y by weight, not row t of it.
template <int G, int VPT, bool kTop>
__global__ void __launch_bounds__(kBlockOf<G>, G > kResident<VPT> ? 1 : kResident<VPT> / kBlockOf<G>) residual_norm(const ResidualNormArgs a) {
    constexpr int B = kBlockOf<G>;
    constexpr int ROWS = B / G;
    constexpr uint32_t kNegate = 0x80008000u;
    // (64 registers a thread do not hold two chunks of everything)
    constexpr bool kEarly = G < 1024 || VPT == 1;
    constexpr int kAhead = kEarly ? 2 : 1;  // rows of a token on their way at a time
    __shared__ alignas(16) float red[3][B / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / G;
    const int i0 = threadIdx.x % G;
    const int C = static_cast<int>(a.K >> 3);
    const int mine = t < a.T ? (C - i0 + G - 1) / G : 0;  // chunks of this thread
    const float K = static_cast<float>(a.K);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    uint4 h[VPT], g[VPT];
    auto load_stream = [&](int i) { h[i] = i < mine ? load(a.h + t * a.ldh + 8 * (i0 + i * G)) : zero; };
    auto load_gate = [&](int i) {
        if (a.gate) g[i] = i < mine ? load(a.gate + t * a.ldg + 8 * (i0 + i * G)) : zero;
    };
    float b[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (kEarly) {
            load_stream(i);
            load_gate(i);
        }
        const uint4 y = !kTop && i < mine ? load(a.y + t * a.ldy + 8 * (i0 + i * G)) : zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) b[i][2 * j] = bf16lo(word(y, j)), b[i][2 * j + 1] = bf16hi(word(y, j));
    }
    if constexpr (kTop) {
        if (mine > 0) {
            const int32_t* rows = a.token_row + t * a.k;
            const float* weights = a.weights ? a.weights + t * a.k : nullptr;
            for (int j = 0; j < a.k; j += kAhead) {
                uint4 y[kAhead][VPT];
                float w[kAhead];
                bool in[kAhead];
#pragma unroll
                for (int l = 0; l < kAhead; ++l) {
                    const int64_t r = j + l < a.k ? rows[j + l] : -1;
                    in[l] = r >= 0 && r < a.R;
                    w[l] = in[l] && weights ? weights[j + l] : 1.0f;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (in[l] && i < mine) y[l][i] = load(a.y + r * a.ldy + 8 * (i0 + i * G));
                }
#pragma unroll
                for (int l = 0; l < kAhead; ++l)
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (in[l] && i < mine) add_scaled(b[i], w[l], y[l][i]);
            }
        }
    }
    if (a.gamma_post) {
        uint4 p[VPT];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            p[i] = i < mine ? load(a.gamma_post + 8 * (i0 + i * G)) : zero;
            squares(b[i], s0, s1);
        }
        const float ss = over_row<G, false>(s0 + s1, red[0]);
        const float inv = 1.0f / sqrtf(ss / K + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            times(b[i], inv);
            times(b[i], p[i]);
        }
    }
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (!kEarly) {
            load_stream(i);
            load_gate(i);
        }
        if (a.gate) times(b[i], g[i]);
        times(b[i], a.branch_scale);
        add_scaled(b[i], a.residual_scale, h[i]);
        squares(b[i], s0, s1);
        if (i < mine) *reinterpret_cast<uint4*>(a.h_out + t * a.ldho + 8 * (i0 + i * G)) = narrow(b[i]);
    }
    if (!a.z && !a.q) return;
    uint4 p[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) p[i] = i < mine ? load(a.gamma + 8 * (i0 + i * G)) : zero;
    const float ss = over_row<G, false>(s0 + s1, red[1]);
    const float inv = -1.0f / sqrtf(ss / K + a.eps);  // (z is negated from here on)
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        times(b[i], inv);
        times(b[i], p[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(b[i][j]));
        if (a.z && i < mine) *reinterpret_cast<uint4*>(a.z + t * a.K + 8 * (i0 + i * G)) = narrow(b[i], kNegate);
    }
    if (!a.q) return;
    m = over_row<G, true>(m, red[2]);
    const float sc = scale_of(m);
    const Divisor d = divisor_of(sc);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (i < mine) *reinterpret_cast<uint2*>(a.q + t * a.ldq + 8 * (i0 + i * G)) = codes_of_negated(b[i], d);
    if (i0 == 0 && t < a.T) a.s[t] = sc;
}

template <int G, int VPT, bool kTop>
cudaError_t launch_as(const ResidualNormArgs& a, cudaStream_t st) {
    constexpr int B = kBlockOf<G>;
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
    return cudaLaunchKernelEx(&cfg, residual_norm<G, VPT, kTop>, a);
}

template <int G, int VPT>
cudaError_t launch(const ResidualNormArgs& a, cudaStream_t st) {
    return a.k > 0 ? launch_as<G, VPT, true>(a, st) : launch_as<G, VPT, false>(a, st);
}

// Chunks of all tokens up to which a thread has one (its serial work is the
// call's latency).  Beyond, two, or four where that was measured to be faster (us,
// two / four chunks a thread):
//   8192 tokens of 4096, y as it is 49.0 / 52.0, two rows by weight 64.1 / 62.7
//   8192 of 1024, two rows 16.1 / 19.3;  of 2048, two rows 42.0 / 41.4
//   4096 of 8192, two rows 94.5 / 84.2;  2048 of 16384, y as it is 87.5 / 73.4
// (one chunk: 8192 of 4096 72.7).
constexpr int64_t kFewChunks = 152 * 1024;

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, cudaStream_t st) {
    const int64_t C = a.K / 8;
    if (a.T * C <= kFewChunks) {
        if (C <= 32) return launch<32, 1>(a, st);
        if (C <= 64) return launch<64, 1>(a, st);
        if (C <= 128) return launch<128, 1>(a, st);
        if (C <= 256) return launch<256, 1>(a, st);
        if (C <= 512) return launch<512, 1>(a, st);
        if (C <= 1024) return launch<1024, 1>(a, st);
    }
    if (C <= (a.k > 0 ? 128 : 512)) {
        if (C <= 64) return launch<32, 2>(a, st);
        if (C <= 128) return launch<64, 2>(a, st);
        if (C <= 256) return launch_as<128, 2, false>(a, st);
        return launch_as<256, 2, false>(a, st);
    }
    if (C <= 256) return launch_as<64, 4, true>(a, st);
    if (C <= 512) return launch_as<128, 4, true>(a, st);
    if (C <= 1024) return launch<256, 4>(a, st);
    if (C <= 2048) return launch<512, 4>(a, st);
    return launch<1024, 4>(a, st);
}

}  // namespace fp8k
