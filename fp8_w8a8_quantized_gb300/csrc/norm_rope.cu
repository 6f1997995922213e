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
// the exact angle, and its upper 32 bits, rounded to fp32's 24, go to sincospif:
// within 2^-26 of a turn (10^-7 radians) at every position, far below the
// output's own rounding.
//
// Bound by memory: every element is read once and written once.  A lane holds
// eight elements of a head, the four pairs that it turns: two runs of four, at
// i and i + rot / 2 (eight consecutive ones where the pairs are neighbours),
// D / 8 lanes (rounded up to a power of two) a head; only the norm needs
// shuffles.  A warp stays with one token for many heads, because its lanes'
// factors are the same in all of them:
//   out_i = (x_i A_i + x_partner B_i) / norm,   A_i = gamma_i cos t,
//                                               B_i = -+ gamma_partner sin t,
// and the heads come through a ring of its own in shared memory, by asynchronous
// copies (loads into registers, two steps at a time: 69 us instead of 64).
//
// Measured: 8192 tokens of 64 + 8 heads of 128 and 8 of values, with norms and
// the cache write: 335 MB in 60 us, 5.6 TB/s, 83% of a plain copy's rate.  What
// is left is instructions: three of four issue slots are taken while all warps
// run, and the last tokens leave SMs idle.  32 tokens: 2.6 us, the launch.
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

constexpr int kDepth = 4;  // steps of a warp on their way (8192 tokens, 72 heads: 2, 4, 8: 66, 63.7, 65.3 us)

// A lane's eight elements: four at `first`, four at `second` (elements).
struct Runs {
    int first, second;
    __device__ uint4 load(const uint16_t* head) const {
        const uint2 a = *reinterpret_cast<const uint2*>(head + first);
        const uint2 b = *reinterpret_cast<const uint2*>(head + second);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    __device__ void copy(uint32_t dst, const uint16_t* head, bool there) const {
        copy_async8(dst, head + first, there);
        copy_async8(dst + 8, head + second, there);
    }
    __device__ void store(uint16_t* head, const uint4& v) const {
        *reinterpret_cast<uint2*>(head + first) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(head + second) = make_uint2(v.z, v.w);
    }
    __device__ void store_codes(uint8_t* head, const uint2& v) const {
        *reinterpret_cast<uint32_t*>(head + first) = v.x;
        *reinterpret_cast<uint32_t*>(head + second) = v.y;
    }
};

// kLanes: lanes of a head (a power of two, kLanes * 8 >= D).  kPairs: pairs
// (2 i, 2 i + 1).  kWhole: all of a head is turned.
template <int kLanes, bool kNorm, bool kPairs, bool kWhole>
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
    const int D = kWhole ? 8 * kLanes : a.D, rot = kWhole ? D : a.rot;
    const bool live = kWhole || chunk < D >> 3;
    const bool turned = kWhole || chunk < rot >> 3;
    Runs at;
    if (kPairs) {
        at.first = 8 * chunk;
        at.second = 8 * chunk + 4;
    } else {  // (what is not turned: two runs as well, of the rest's halves)
        const int from = turned ? 0 : rot, size = turned ? rot : D - rot;
        at.first = from + 4 * (chunk - (from >> 3));
        at.second = at.first + (size >> 1);
    }

    // steps of kHeads heads: the queries', the keys', the values'
    const int steps_q = (a.Hq + kHeads - 1) / kHeads, steps_k = (a.Hkv + kHeads - 1) / kHeads;
    const int steps = steps_q + steps_k + (a.k_cache ? steps_k : 0);
    const int per = (steps + slices - 1) / slices;
    const int begin = slice * per, end = min(steps, begin + per);

    // The steps' elements come through a ring in shared memory, kDepth steps
    // ahead, each lane's by its own copies.
    __shared__ __align__(16) uint8_t ring_of[kThreads / 32][kDepth][512];
    const uint32_t ring = smem_u32(ring_of[threadIdx.x >> 5]) + 16 * lane;
    auto fetch = [&](int step) {
        const uint32_t to = ring + (step - begin) % kDepth * 512;
        if (step < steps_q) {
            const int head = step * kHeads + sub;
            at.copy(to, a.q + t * a.ldq + head * D, live && head < a.Hq);
        } else if (step < end) {
            const bool key = step < steps_q + steps_k;
            const int head = (step - steps_q - (key ? 0 : steps_k)) * kHeads + sub;
            if (key) at.copy(to, a.k + t * a.ldk + head * D, live && head < a.Hkv);
            else copy_async16(to, a.v + t * a.ldv + head * D + chunk * 8, live && head < a.Hkv);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        if (begin + i < end) fetch(begin + i);
        else copy_commit();
    }
    auto arrived = [&](int step) {
        copy_wait<kDepth - 1>();
        const uint4 u = ld_shared16(ring + (step - begin) % kDepth * 512);
        __syncwarp();
        if (step + kDepth < end) fetch(step + kDepth);
        else copy_commit();
        return u;
    };

    const int64_t slot = a.k_cache ? (a.slot ? a.slot[t] : t) : -1;
    const bool store = slot >= 0 && slot < a.n_slots;
    const float inv_d = 1.0f / static_cast<float>(D);

    // this lane's sines and cosines, of its four pairs
    float co[4], si[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) co[i] = 1.0f, si[i] = 0.0f;
    if (turned && live) {
        const uint64_t position = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t turns = position * a.turns[4 * chunk + i];
            const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
            sincospif(x, &si[i], &co[i]);
        }
    }
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {  // queries, keys
        const int off = kind ? steps_q : 0;
        const int lo = max(begin, off) - off, hi = min(end, off + (kind ? steps_k : steps_q)) - off;
        if (lo >= hi) continue;
        const int heads = kind ? a.Hkv : a.Hq;
        uint16_t* dst = kind ? (a.k_out ? a.k_out + t * a.ldko : nullptr) : a.q_out + t * a.ldqo;
        const uint16_t* gamma = kind ? a.gamma_k : a.gamma_q;
        const bool normed = kNorm && gamma;
        float A[8], B[8];  // of elements 0-3 and 4-7
        {
            float g[8];
            if (normed && live) {
                widen8(at.load(gamma), g);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // (what is not turned: x A + 0 (-0) keeps even a zero's sign)
                const int pair = kPairs ? i >> 1 : i & 3, other = kPairs ? i ^ 1 : i ^ 4;
                const bool low = kPairs ? !(i & 1) : i < 4;
                A[i] = g[i] * co[pair];
                B[i] = !turned ? -0.0f : low ? -g[other] * si[pair] : g[other] * si[pair];
            }
        }
        for (int step = lo; step < hi; ++step) {
            const uint4 u = arrived(off + step);
            const int head = step * kHeads + sub;
            float x[8];
            widen8(u, x);
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
                const int p = kPairs ? i + 1 : i ^ 4, q = kPairs ? i : (i ^ 4) + 1;
                const float z0 = turned ? x[p] : 0.0f, z1 = turned ? x[q] : 0.0f;
                mul2(y[i], y[i + 1], x[i], x[i + 1], A[i], A[i + 1]);
                fma2(y[i], y[i + 1], z0, z1, B[i], B[i + 1]);
                if (kNorm) mul2(y[i], y[i + 1], y[i], y[i + 1], inv, inv);
            }
            const uint4 o = make_uint4(narrow2(y[0], y[1]), narrow2(y[2], y[3]), narrow2(y[4], y[5]),
                                       narrow2(y[6], y[7]));
            if (!live || head >= heads) continue;
            if (dst) at.store(dst + head * D, o);
            if (kind && store) {
                const float s = a.k_scale[head * a.scale_stride];
                at.store_codes(a.k_cache + (slot * a.Hkv + head) * D, quant8<false>(o, divisor_of(s)));
            }
        }
    }
    // values: to the cache as they are
    const int off = steps_q + steps_k;
    for (int step = max(begin, off) - off; store && step < end - off; ++step) {
        const uint4 u = arrived(off + step);
        const int head = step * kHeads + sub;
        if (!live || head >= a.Hkv) continue;
        const float s = a.v_scale[head * a.scale_stride];
        *reinterpret_cast<uint2*>(a.v_cache + (slot * a.Hkv + head) * D + chunk * 8) =
            quant8<false>(u, divisor_of(s));
    }
    copy_wait<0>();  // (values of a token without a slot were asked for all the same)
}

template <int kLanes, bool kWhole>
auto kernel_of(bool norm, bool pairs) {
    return norm ? (pairs ? qk_norm_rope<kLanes, true, true, kWhole> : qk_norm_rope<kLanes, true, false, kWhole>)
                : (pairs ? qk_norm_rope<kLanes, false, true, kWhole> : qk_norm_rope<kLanes, false, false, kWhole>);
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
    // (a lane beyond D / 8 has nothing to turn either)
    auto kernel = a.rot == a.D && a.D == 8 * kLanes ? kernel_of<kLanes, true>(norm, a.pairs)
                                                    : kernel_of<kLanes, false>(norm, a.pairs);
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
