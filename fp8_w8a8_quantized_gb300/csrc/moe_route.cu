// Routing: each token's best experts, their weights, and the rows that the
// (token, expert) pairs make, sorted by expert and by token within one.
//
//   ids[t, j]     = expert of the j-th largest logit, the lower number first
//   weights[t, j] = scale exp(l - max) / sum exp(l - max)
//   rows          = the pairs in the order (expert, token)
//
// Two launches.  choose: a warp a token, its logits in registers (E / 32 a
// lane), as unsigned numbers whose order is the logits' own; k rounds of a
// warp maximum and the lowest expert that has it (two redux instructions).
// Tokens are cut into as many parts as there are CTAs, and each CTA leaves how
// many pairs of its part chose each expert.  place: the row of a pair is the
// pairs of lower experts + those of earlier parts + those before it in its own
// part.  Every CTA adds up the first two for itself from the parts' counts,
// and its warps number their pairs 32 at a time (match.sync).  Counts are
// whole numbers, so nothing depends on an order of arrival.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxParts = 152;  // parts of the tokens: a CTA an SM

// An unsigned number in the order of the floats; 0 for what is switched off
// (NaN and -infinity, whose own number would be 0x007FFFFF).
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // (both zeros alike)
    return v > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float logit(const float* p) { return *p; }
__device__ __forceinline__ float logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// tokens [first, last) of a part, of a warp within it
__device__ __forceinline__ void share(int64_t n, int parts, int part, int64_t* first, int64_t* last) {
    const int64_t per = n / parts, rem = n % parts;
    *first = part * per + min(static_cast<int64_t>(part), rem);
    *last = *first + per + (part < rem ? 1 : 0);
}

template <typename Logit, int kPerLane>
__global__ void __launch_bounds__(kThreads)
    route_choose(const Logit* logits, int64_t ld, int64_t T, int E, int k, bool renorm, float scale,
                 int32_t* ids, float* weights, int32_t* counts) {
    __shared__ int32_t count[kPerLane * 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
    __syncthreads();
    int64_t first, last;
    share(T, gridDim.x, blockIdx.x, &first, &last);
    for (int64_t t = first + warp; t < last; t += kWarps) {
        uint32_t o[kPerLane];
        uint32_t mine = 0;  // this lane's largest
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = i * 32 + lane;
            o[i] = e < E ? order_of(logit(logits + t * ld + e)) : 0u;
            mine = max(mine, o[i]);
        }
        float best = 0.0f, total = 0.0f;
        int got_id = -1;      // lane j keeps the token's j-th expert
        float got_w = 0.0f;
        for (int j = 0; j < k; ++j) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, mine);
            if (top == 0) break;
            int at = E;  // the lane's lowest expert with that logit
#pragma unroll
            for (int i = kPerLane - 1; i >= 0; --i)
                if (o[i] == top) at = i * 32 + lane;
            const int id = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<unsigned>(at)));
            const float v = value_of(top);
            if (j == 0) {
                best = v;
                if (!renorm) {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i)
                        if (o[i]) s += expf(value_of(o[i]) - best);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
                    total = s;
                }
            }
            const float w = expf(v - best);
            if (renorm) total += w;
            if (lane == j) {
                got_id = id;
                got_w = w;
            }
            mine = 0;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (i * 32 + lane == id) o[i] = 0;
                mine = max(mine, o[i]);
            }
        }
        if (lane < k) {
            ids[t * k + lane] = got_id;
            weights[t * k + lane] = got_id < 0 ? 0.0f : got_w / total * scale;
            if (got_id >= 0) atomicAdd(&count[got_id], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] = count[e];
}

// Sums of the elements before each of a CTA's threads, and of all.
__device__ __forceinline__ int32_t before(int32_t v, int32_t* all, int32_t* warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += u;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int32_t sum = 0;
    *all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) sum += warp_sums[w];
        *all += warp_sums[w];
    }
    __syncthreads();
    return sum + incl - v;
}

__global__ void __launch_bounds__(kThreads)
    route_place(const int32_t* ids, const int32_t* counts, int parts, int64_t T, int E, int k,
                int32_t* offsets, int32_t* row_token, int32_t* token_row) {
    extern __shared__ int32_t shared[];
    int32_t* next = shared;               // [kWarps][E]: a warp's pairs, then its next row of each expert
    int32_t* base = shared + kWarps * E;  // [E]: pairs of an expert, then its first row in this part
    int32_t* prior = base + E;            // [E]: its pairs in earlier parts
    __shared__ int32_t warp_sums[kWarps];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x;
    for (int i = threadIdx.x; i < kWarps * E; i += kThreads) next[i] = 0;
    for (int e = warp; e < E; e += kWarps) {
        int32_t all = 0, mine = 0;
        for (int c = lane; c < parts; c += 32) {
            const int32_t n = counts[static_cast<int64_t>(e) * parts + c];
            all += n;
            if (c < part) mine += n;
        }
        all = __reduce_add_sync(0xFFFFFFFFu, all);
        mine = __reduce_add_sync(0xFFFFFFFFu, mine);
        if (lane == 0) {
            base[e] = all;
            prior[e] = mine;
        }
    }
    __syncthreads();
    int32_t rows = 0;  // of the experts so far
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        int32_t all;
        const int32_t first = rows + before(e < E ? base[e] : 0, &all, warp_sums);
        if (e < E) {
            base[e] = first + prior[e];
            if (part == 0) offsets[e] = first;
        }
        rows += all;
    }
    if (part == 0 && threadIdx.x == 0) offsets[E] = rows;
    // the pairs of this part, of this warp
    int64_t t0, t1, w0, w1;
    share(T, parts, part, &t0, &t1);
    share(t1 - t0, kWarps, warp, &w0, &w1);
    const int64_t p0 = (t0 + w0) * k, p1 = (t0 + w1) * k;
    for (int64_t p = p0 + lane; p < p1; p += 32) {
        const int e = ids[p];
        if (e >= 0) atomicAdd(&next[warp * E + e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int32_t at = base[e];
        for (int w = 0; w < kWarps; ++w) {
            const int32_t n = next[w * E + e];
            next[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t q = p0; q < p1; q += 32) {
        const int64_t p = q + lane;
        const int e = p < p1 ? ids[p] : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        int32_t row = -1;
        if (e >= 0) {
            row = next[warp * E + e] + __popc(same & ((1u << lane) - 1u));
            row_token[row] = static_cast<int32_t>(p / k);
        }
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) next[warp * E + e] += __popc(same);
        __syncwarp();
        if (p < p1) token_row[p] = row;
    }
    for (int64_t r = rows + static_cast<int64_t>(part) * kThreads + threadIdx.x; r < T * k;
         r += static_cast<int64_t>(parts) * kThreads)
        row_token[r] = -1;
}

int parts_of(int64_t T) {  // a token a warp at least
    const int64_t n = (T + kWarps - 1) / kWarps;
    return static_cast<int>(n < 1 ? 1 : n < kMaxParts ? n : kMaxParts);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Logit>
cudaError_t launch_choose(const RouteArgs& a, int parts, cudaStream_t st) {
    const Logit* l = static_cast<const Logit*>(a.logits);
    auto go = [&](auto kernel) {
        return launch(kernel, parts, 0, st, l, a.ld, a.T, a.E, a.k, a.renorm, a.scale, a.ids, a.weights, a.workspace);
    };
    if (a.E <= 32) return go(route_choose<Logit, 1>);
    if (a.E <= 64) return go(route_choose<Logit, 2>);
    if (a.E <= 128) return go(route_choose<Logit, 4>);
    if (a.E <= 256) return go(route_choose<Logit, 8>);
    if (a.E <= 512) return go(route_choose<Logit, 16>);
    return go(route_choose<Logit, 32>);
}

}  // namespace

size_t moe_route_workspace(int64_t T, int64_t E, int64_t k) {
    (void)k;
    return sizeof(int32_t) * static_cast<size_t>(E) * parts_of(T);
}

cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t st) {
    const int parts = parts_of(a.T);
    const cudaError_t e = a.fp32 ? launch_choose<float>(a, parts, st) : launch_choose<__nv_bfloat16>(a, parts, st);
    if (e != cudaSuccess) return e;
    return launch(route_place, parts, sizeof(int32_t) * (kWarps + 2) * a.E, st, a.ids, a.workspace, parts, a.T, a.E, a.k,
                  a.offsets, a.row_token, a.token_row);
}

}  // namespace fp8k
