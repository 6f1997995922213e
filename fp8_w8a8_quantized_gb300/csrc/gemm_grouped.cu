// Products of each expert's rows with that expert's weights, rows sorted by
// expert with bounds known on the GPU alone:
//   a[r, n] = ((sum_k e4m3(xq[r, k]) e4m3(wq[e, n, k])) s_tok[r]) s_w[e, n]
//   y = bf16(a), or bf16(silu(a[:, n]) a[:, n + N / 2])
//
// Simple form: a 32 x 32 tile of outputs a CTA, codes converted to fp32 in
// shared memory, sums in fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr int kTile = 32;
constexpr int kDepth = 64;
constexpr int kThreads = 256;

__device__ __forceinline__ float value(uint8_t code) {
    __nv_fp8_e4m3 v;
    v.__x = code;
    return static_cast<float>(v);
}

__global__ void __launch_bounds__(kThreads)
    grouped_simple(const uint8_t* xq, const float* s_tok, const uint8_t* wq,
                   const float* s_w, const int32_t* offsets, int R, int N, int K, bool swiglu,
                   __nv_bfloat16* y) {
    __shared__ float xs[kTile][kDepth + 1], ws[2][kTile][kDepth + 1];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int e = blockIdx.y;
    const int begin = min(max(offsets[e], 0), R), end = min(max(offsets[e + 1], begin), R);
    const int F = swiglu ? N / 2 : N;
    const int n0 = blockIdx.x * kTile;
    const int c = threadIdx.x % kTile, r0 = threadIdx.x / kTile;
    for (int m0 = begin; m0 < end; m0 += kTile) {
        float acc[2][4] = {};
        for (int k0 = 0; k0 < K; k0 += kDepth) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
                const int r = i / kDepth, k = i % kDepth;
                const bool in = k0 + k < K;
                xs[r][k] = in && m0 + r < end ? value(xq[static_cast<int64_t>(m0 + r) * K + k0 + k]) : 0.0f;
                for (int h = 0; h < (swiglu ? 2 : 1); ++h)
                    ws[h][r][k] = in && n0 + r < F
                                      ? value(wq[(static_cast<int64_t>(e) * N + h * F + n0 + r) * K + k0 + k])
                                      : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kDepth; ++k)
                for (int h = 0; h < (swiglu ? 2 : 1); ++h)
                    for (int i = 0; i < 4; ++i) acc[h][i] += xs[r0 + 8 * i][k] * ws[h][c][k];
        }
        const int n = n0 + c;
        if (n < F)
            for (int i = 0; i < 4; ++i) {
                const int r = m0 + r0 + 8 * i;
                if (r >= end) continue;
                float v = acc[0][i] * s_tok[r] * s_w[static_cast<int64_t>(e) * N + n];
                if (swiglu) v = v / (1.0f + expf(-v)) * (acc[1][i] * s_tok[r] * s_w[static_cast<int64_t>(e) * N + F + n]);
                y[static_cast<int64_t>(r) * F + n] = __float2bfloat16_rn(v);
            }
    }
}

}  // namespace

size_t gemm_grouped_workspace(int64_t E, int64_t R, int64_t N, int64_t K) {
    (void)E, (void)R, (void)N, (void)K;
    return 0;
}

int64_t gemm_grouped_zero_words() { return 0; }

cudaError_t prepare_gemm_grouped() { return cudaSuccess; }

cudaError_t launch_gemm_grouped(const GroupedArgs& a, cudaStream_t st) {
    const int F = a.swiglu ? a.N / 2 : a.N;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((F + kTile - 1) / kTile, a.E);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, grouped_simple, a.xq, a.s_tok, a.wq, a.s_w, a.offsets, a.R, a.N, a.K, a.swiglu,
                              static_cast<__nv_bfloat16*>(a.y));
}

}  // namespace fp8k
