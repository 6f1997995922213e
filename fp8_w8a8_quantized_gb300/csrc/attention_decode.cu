// Attention over packed prompts and over the paged FP8 cache:
//   out = softmax(scale q k^T) v over the keys that a query may see, zero
//   where it may see none.
// One warp per query and head, one pass over the keys with the running
// maximum m and sum l of the softmax and the running output o, all in fp32:
//   m' = max(m, s), o' = o e^(m - m') + e^(s - m') v, l' = l e^(m - m') + e^(s - m').
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void widen4(const uint2& u, float (&f)[4]) {
    f[0] = bf16lo(u.x), f[1] = bf16hi(u.x), f[2] = bf16lo(u.y), f[3] = bf16hi(u.y);
}

__device__ __forceinline__ void e4m3x4(uint32_t u, float (&f)[4]) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(u), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(u >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

struct Row {
    float m = -INFINITY, l = 0.0f, o[4] = {};
    __device__ void add(const float (&q)[4], const float (&k)[4], const float (&v)[4], float c) {
        float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        s *= c;
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.0f : exp2f(m - top);
        const float p = exp2f(s - top);
        l = l * keep + p;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + p * v[i];
        m = top;
    }
    __device__ void write(uint16_t* dst, float c) const {
        const float inv = l > 0.0f || l != l ? c / l : 0.0f;
        const __nv_bfloat162 a = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                    *reinterpret_cast<const uint32_t*>(&b));
    }
};

__global__ void __launch_bounds__(kThreads) attention_decode(const DecodeArgs a) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t b = w / a.Hq;
    const int h = static_cast<int>(w - b * a.Hq), hk = h / (a.Hq / a.Hkv);
    if (b >= a.B) return;
    const int lane = lane_id();
    const bool on = lane * 4 < a.D;
    const int64_t room = a.width * a.page;
    const int64_t len = a.lens[b] < room ? a.lens[b] : room;
    const float c = a.scale * kLog2e * a.k_scale[hk * a.scale_stride];
    float q[4] = {};
    if (on) widen4(*reinterpret_cast<const uint2*>(a.q + b * a.ldq + h * a.D + lane * 4), q);
    Row r;
    for (int64_t j = 0; j < len; ++j) {
        const int64_t id = a.table[(j < a.prefix ? 0 : b) * a.ld_table + j / a.page];
        if (id < 0 || id >= a.n_pages) continue;
        const int64_t off = ((id * a.page + j % a.page) * a.Hkv + hk) * a.D + lane * 4;
        float k[4] = {}, v[4] = {};
        if (on) {
            e4m3x4(*reinterpret_cast<const uint32_t*>(a.k_cache + off), k);
            e4m3x4(*reinterpret_cast<const uint32_t*>(a.v_cache + off), v);
        }
        r.add(q, k, v, c);
    }
    if (on) r.write(a.out + b * a.ldo + h * a.D + lane * 4, a.v_scale[hk * a.scale_stride]);
}

template <typename Args>
cudaError_t launch(void (*kernel)(Args), int64_t warps, cudaStream_t st, const Args& a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t attention_decode_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) {
    return 0;
}

cudaError_t launch_attention_decode(const DecodeArgs& a, cudaStream_t st) {
    return launch(attention_decode, a.B * a.Hq, st, a);
}

}  // namespace fp8k
