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
// factors are the same in all of them:
//   out_i = (x_i A_i + x_partner B_i) / norm,   A_i = gamma_i cos t,
//                                               B_i = -+ gamma_partner sin t,
// and takes kBatch heads' loads at a time.
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

constexpr int kBatch = 2;  // heads' loads of a lane on their way (four CTAs an SM; four heads, three CTAs: 4% slower)

__device__ __forceinline__ void gamma8(const uint16_t* gamma, int chunk, bool live, float (&g)[8]) {
    if (gamma && live) {
        widen8(__ldg(reinterpret_cast<const uint4*>(gamma + chunk * 8)), g);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 1.0f;
    }
}

// kLanes: lanes of a head (a power of two, kLanes * 8 >= D).
template <int kLanes, bool kNorm, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope(const QkNormRopeArgs a, int slices) {
    pdl_launch_dependents();
    pdl_wait_primary();
    constexpr int kHeads = 32 / kLanes;  // heads of a warp at a time
    const int lane = lane_id();
    const int chunk = lane & (kLanes - 1), sub = lane / kLanes;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = w / slices;
    if (t >= a.T) return;
    const int slice = static_cast<int>(w - t * slices);
    const bool live = chunk < a.D >> 3;
    const int half = a.rot >> 4;  // chunks of half the rotated part (pairs d, d + rot / 2)
    const bool turned = chunk < 2 * half;
    const int partner = kPairs || !turned ? chunk : chunk < half ? chunk + half : chunk - half;
    const int from = (lane & ~(kLanes - 1)) + partner;

    // this lane's sines and cosines: eight pairs, or the four within its chunk
    float co[8], si[8];
    // (what is not turned: x A + 0 (-0) keeps even a zero's sign)
#pragma unroll
    for (int i = 0; i < 8; ++i) co[i] = 1.0f, si[i] = -0.0f;
    if (turned) {
        const uint64_t position = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t]));
        const int base = kPairs ? chunk * 4 : (chunk < half ? chunk : chunk - half) * 8;
#pragma unroll
        for (int i = 0; i < (kPairs ? 4 : 8); ++i) {
            const uint64_t turns = position * a.turns[base + i];
            const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
            float s, c;
            sincospif(x, &s, &c);
            if (kPairs) {
                co[2 * i] = co[2 * i + 1] = c;
                si[2 * i] = -s;
                si[2 * i + 1] = s;
            } else {
                co[i] = c;
                si[i] = chunk < half ? -s : s;
            }
        }
    }
    const int64_t slot = a.k_cache ? (a.slot ? a.slot[t] : t) : -1;
    const bool store = slot >= 0 && slot < a.n_slots;
    const float inv_d = 1.0f / static_cast<float>(a.D);

    // steps of kHeads heads: the queries', the keys', the values'
    const int steps_q = (a.Hq + kHeads - 1) / kHeads, steps_k = (a.Hkv + kHeads - 1) / kHeads;
    const int steps = steps_q + steps_k + (store ? steps_k : 0);
    const int per = (steps + slices - 1) / slices;
    const int begin = slice * per, end = min(steps, begin + per);

#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {  // queries, keys
        const int off = kind ? steps_q : 0;
        const int lo = max(begin, off) - off, hi = min(end, off + (kind ? steps_k : steps_q)) - off;
        if (lo >= hi) continue;
        const int heads = kind ? a.Hkv : a.Hq;
        const uint16_t* src = (kind ? a.k + t * a.ldk : a.q + t * a.ldq) + chunk * 8;
        uint16_t* dst = kind ? (a.k_out ? a.k_out + t * a.ldko + chunk * 8 : nullptr)
                             : a.q_out + t * a.ldqo + chunk * 8;
        const uint16_t* gamma = kind ? a.gamma_k : a.gamma_q;
        const bool normed = kNorm && gamma;
        float A[8], B[8];
        gamma8(kNorm ? gamma : nullptr, chunk, live, A);
        gamma8(kNorm ? gamma : nullptr, partner, live, B);
#pragma unroll
        for (int i = 0; i < 8; ++i) A[i] *= co[i];
        if (kPairs) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float other = B[i];
                B[i] = turned ? B[i + 1] * si[i] : si[i];
                B[i + 1] = turned ? other * si[i + 1] : si[i + 1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) B[i] = turned ? B[i] * si[i] : si[i];
        }
        for (int step = lo; step < hi; step += kBatch) {
            uint4 u[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int head = (step + j) * kHeads + sub;
                u[j] = make_uint4(0, 0, 0, 0);
                if (live && step + j < hi && head < heads)
                    u[j] = *reinterpret_cast<const uint4*>(src + head * a.D);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (step + j >= hi) break;  // (the whole warp)
                const int head = (step + j) * kHeads + sub;
                float x[8], z[8];
                widen8(u[j], x);
                if (kPairs) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = turned ? x[i ^ 1] : 0.0f;
                } else {
                    uint4 v = make_uint4(__shfl_sync(0xFFFFFFFFu, u[j].x, from),
                                         __shfl_sync(0xFFFFFFFFu, u[j].y, from),
                                         __shfl_sync(0xFFFFFFFFu, u[j].z, from),
                                         __shfl_sync(0xFFFFFFFFu, u[j].w, from));
                    if (!turned) v = make_uint4(0, 0, 0, 0);
                    widen8(v, z);
                }
                float inv = 1.0f;
                if (kNorm) {
                    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) fma2(s0, s1, x[i], x[i + 1], x[i], x[i + 1]);
                    float ss = s0 + s1;
#pragma unroll
                    for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
                    if (normed) inv = rsqrtf(fmaf(ss, inv_d, a.eps));
                }
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    mul2(y[i], y[i + 1], x[i], x[i + 1], A[i], A[i + 1]);
                    fma2(y[i], y[i + 1], z[i], z[i + 1], B[i], B[i + 1]);
                    if (kNorm) mul2(y[i], y[i + 1], y[i], y[i + 1], inv, inv);
                }
                const uint4 o = make_uint4(narrow2(y[0], y[1]), narrow2(y[2], y[3]), narrow2(y[4], y[5]),
                                           narrow2(y[6], y[7]));
                if (!live || head >= heads) continue;
                if (dst) *reinterpret_cast<uint4*>(dst + head * a.D) = o;
                if (kind && store) {
                    const float s = __ldg(a.k_scale + head * a.scale_stride);
                    *reinterpret_cast<uint2*>(a.k_cache + (slot * a.Hkv + head) * a.D + chunk * 8) =
                        quant8<false>(o, divisor_of(s));
                }
            }
        }
    }
    // values: to the cache as they are
    const int off = steps_q + steps_k;
    for (int step = max(begin, off) - off; step < end - off; step += kBatch) {
        uint4 u[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int head = (step + j) * kHeads + sub;
            u[j] = make_uint4(0, 0, 0, 0);
            if (live && step + j < end - off && head < a.Hkv)
                u[j] = *reinterpret_cast<const uint4*>(a.v + t * a.ldv + head * a.D + chunk * 8);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int head = (step + j) * kHeads + sub;
            if (!live || step + j >= end - off || head >= a.Hkv) continue;
            const float s = __ldg(a.v_scale + head * a.scale_stride);
            *reinterpret_cast<uint2*>(a.v_cache + (slot * a.Hkv + head) * a.D + chunk * 8) =
                quant8<false>(u[j], divisor_of(s));
        }
    }
}

template <int kLanes>
cudaError_t launch_lanes(const QkNormRopeArgs& a, int num_sms, cudaStream_t st) {
    constexpr int kHeads = 32 / kLanes;
    const int steps = (a.Hq + kHeads - 1) / kHeads + (a.Hkv + kHeads - 1) / kHeads * (a.k_cache ? 2 : 1);
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
