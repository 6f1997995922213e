// Norms of queries and keys for each head, with the rotation of their
// positions, and the FP8 cache write of the rotated keys and the values, in
// one pass over a step's fused projection:
//
//   y_d = x_d / sqrt(mean_d x_d^2 + eps) * gamma_d         (or y = x)
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//   out = bf16_rn(y),  cache[slot, h, :] = E4M3_rn_sat(out / scale[h])
//
// all in fp32 with one rounding to bf16.  The angle t = position * frequency
// loses its digits in fp32 at far positions, so frequencies come as 64-bit
// fractions of a turn: the integer product position * turns, modulo 2^64, is
// the exact angle, its upper 32 bits are within 2^-32 of a turn, and
// sincospif takes them from there.
//
// Bound by memory: every element is read once and written once.  A lane holds
// eight consecutive elements of a head (one 16-byte access), D / 8 lanes
// (rounded up to a power of two) a head, so norm and rotation need only
// shuffles.  A warp stays with one token for many heads, because its lanes'
// sines and cosines are the same in all of them: at 80 heads a token they are
// a few instructions a head.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void widen8(const uint4& u, float (&f)[8]) {
    f[0] = bf16lo(u.x), f[1] = bf16hi(u.x), f[2] = bf16lo(u.y), f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z), f[5] = bf16hi(u.z), f[6] = bf16lo(u.w), f[7] = bf16hi(u.w);
}

__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// kLanes: lanes of a head (a power of two, kLanes * 8 >= D).
template <int kLanes, bool kNorm, bool kPairs>
__global__ void __launch_bounds__(kThreads) qk_norm_rope(const QkNormRopeArgs a, int slices) {
    pdl_launch_dependents();
    pdl_wait_primary();
    constexpr int kHeads = 32 / kLanes;  // heads of a warp at a time
    const int lane = lane_id();
    const int chunk = lane & (kLanes - 1), sub = lane / kLanes;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = w / slices;
    if (t >= a.T) return;
    const int slice = static_cast<int>(w - t * slices);
    const int chunks = a.D >> 3;
    const bool live = chunk < chunks;
    const int half = a.rot >> 4;  // chunks of half the rotated part (pairs d, d + rot / 2)
    const bool turned = kPairs ? chunk < 2 * half : live && chunk < 2 * half;
    const int partner = kPairs || !turned ? chunk : chunk < half ? chunk + half : chunk - half;

    // this lane's sines and cosines: eight pairs, or the four within its chunk
    float co[8], si[8];
    if (turned) {
        const uint64_t position = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t]));
        const int base = kPairs ? chunk * 4 : (chunk < half ? chunk : chunk - half) * 8;
#pragma unroll
        for (int i = 0; i < (kPairs ? 4 : 8); ++i) {
            const uint64_t turns = position * a.turns[base + i];
            const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
            sincospif(x, &si[i], &co[i]);
            if (!kPairs && chunk < half) si[i] = -si[i];
        }
    }
    const int64_t slot = a.k_cache ? (a.slot ? a.slot[t] : t) : -1;
    const bool store = slot >= 0 && slot < a.n_slots;
    const int rows = a.Hq + a.Hkv + (store ? a.Hkv : 0);  // queries, keys, then values
    const int steps = (rows + kHeads - 1) / kHeads;
    const int per = (steps + slices - 1) / slices;
    const int end = min(steps, (slice + 1) * per);

    const float inv_d = 1.0f / static_cast<float>(a.D);
    for (int step = slice * per; step < end; ++step) {
        const int row = step * kHeads + sub;
        const bool is_q = row < a.Hq, is_v = row >= a.Hq + a.Hkv;
        const int head = is_q ? row : is_v ? row - a.Hq - a.Hkv : row - a.Hq;
        const bool on = live && row < rows;
        const uint16_t* src = is_q ? a.q + t * a.ldq : is_v ? a.v + t * a.ldv : a.k + t * a.ldk;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (on) u = *reinterpret_cast<const uint4*>(src + head * a.D + chunk * 8);
        uint4 o = u;
        if (!is_v || kHeads > 1) {  // (lanes of a value head only join the shuffles)
            float x[8];
            widen8(u, x);
            const uint16_t* gamma = is_q ? a.gamma_q : a.gamma_k;
            const bool normed = kNorm && gamma && !is_v;
            float inv = 1.0f;
            if (kNorm) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
                if (normed) inv = 1.0f / sqrtf(fmaf(ss, inv_d, a.eps));
            }
            float y[8];
            if (normed && on) {
                float g[8];
                widen8(__ldg(reinterpret_cast<const uint4*>(gamma + chunk * 8)), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i] * inv * g[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i];
            }
            float r[8];
            if (kPairs) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[2 * i] = y[2 * i] * co[i] - y[2 * i + 1] * si[i];
                    r[2 * i + 1] = y[2 * i + 1] * co[i] + y[2 * i] * si[i];
                }
            } else {
                const int from = (lane & ~(kLanes - 1)) + partner;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float z = __shfl_sync(0xFFFFFFFFu, y[i], from);
                    r[i] = y[i] * co[i] + z * si[i];
                }
            }
            if (!is_v) {
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = r[i];
                }
                o = make_uint4(narrow2(y[0], y[1]), narrow2(y[2], y[3]), narrow2(y[4], y[5]),
                               narrow2(y[6], y[7]));
            }
        }
        if (!on) continue;
        if (is_q) {
            *reinterpret_cast<uint4*>(a.q_out + t * a.ldqo + head * a.D + chunk * 8) = o;
            continue;
        }
        if (!is_v && a.k_out)
            *reinterpret_cast<uint4*>(a.k_out + t * a.ldko + head * a.D + chunk * 8) = o;
        if (store) {
            const float s = __ldg((is_v ? a.v_scale : a.k_scale) + head * a.scale_stride);
            uint8_t* dst = is_v ? a.v_cache : a.k_cache;
            *reinterpret_cast<uint2*>(dst + (slot * a.Hkv + head) * a.D + chunk * 8) =
                quant8<false>(o, divisor_of(s));
        }
    }
}

template <int kLanes>
cudaError_t launch_lanes(const QkNormRopeArgs& a, int num_sms, cudaStream_t st) {
    const int rows = a.Hq + a.Hkv * (a.k_cache ? 2 : 1);
    const int steps = (rows + 32 / kLanes - 1) / (32 / kLanes);
    // Few tokens: a token's heads are divided among warps until the SMs have
    // 16 warps each or a warp has one step left.
    int slices = 1;
    while (slices < steps && a.T * slices < static_cast<int64_t>(num_sms) * 16) slices *= 2;
    const int64_t warps = a.T * slices;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool norm = a.gamma_q || a.gamma_k;
    auto kernel = norm ? (a.pairs ? qk_norm_rope<kLanes, true, true> : qk_norm_rope<kLanes, true, false>)
                       : (a.pairs ? qk_norm_rope<kLanes, false, true> : qk_norm_rope<kLanes, false, false>);
    return cudaLaunchKernelEx(&cfg, kernel, a, slices);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& a, int num_sms, cudaStream_t st) {
    const int chunks = a.D >> 3;
    if (chunks <= 2) return launch_lanes<2>(a, num_sms, st);
    if (chunks <= 4) return launch_lanes<4>(a, num_sms, st);
    if (chunks <= 8) return launch_lanes<8>(a, num_sms, st);
    if (chunks <= 16) return launch_lanes<16>(a, num_sms, st);
    return launch_lanes<32>(a, num_sms, st);
}

}  // namespace fp8k
