// Routing: each token's best experts, their weights, and the rows that the
// (token, expert) pairs make, sorted by expert and by token within one.
//
//   ids[t, j]     = expert of the j-th largest logit, the lower number first
//   weights[t, j] = scale exp(l - max) / sum exp(l - max)
//   rows          = the pairs in the order (expert, token)
//
// A warp takes a token, its logits in registers (E / 32 a lane) as unsigned
// numbers whose order is the logits' own: k rounds of a warp maximum and the lowest
// expert that has it (two redux instructions).  The tokens are cut into parts, a
// CTA each, which counts how many pairs of its part chose each expert.  The row of
// a pair is the pairs of lower experts + those of earlier parts + those before it
// in its own part, which 8 of the CTA's warps number 32 pairs at a time
// (match.sync).  Counts are whole numbers: nothing depends on an order of arrival.
//
// Up to kClusterTokens tokens it is one launch of one cluster, whose CTAs read one
// another's counts through distributed shared memory; beyond, two launches with
// the counts in the workspace (choose, place).  Small calls are bound by latency
// (launch, logits, k rounds, numbering), large ones by the rounds' instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr int kPlacers = 8;             // warps that number the pairs of a part
constexpr int kMaxParts = 152;          // parts of two launches: a CTA an SM
constexpr int kClusterParts = 8;
constexpr int64_t kClusterTokens = 1024;

// Threads of a CTA: as many as the registers for kPerLane logits a lane allow.
template <int kPerLane>
constexpr int kThreadsOf = kPerLane <= 8 ? 1024 : 512;

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

struct Route {
    const void* logits;
    int64_t ld, T;
    int E, k;
    bool renorm;
    float scale;
    int32_t* ids;
    float* weights;
    int32_t *offsets, *row_token, *token_row;
    int32_t* counts;  // [parts][E], with two launches
};

// The experts of tokens first .. last - 1, counted in `count`.
template <typename Logit, int kPerLane>
__device__ __forceinline__ void choose(const Route& a, int64_t first, int64_t last, int32_t* count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Logit* logits = static_cast<const Logit*>(a.logits);
    for (int64_t t = first + warp; t < last; t += kThreadsOf<kPerLane> / 32) {
        float v[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = i * 32 + lane;
            v[i] = e < a.E ? logit(logits + t * a.ld + e) : -INFINITY;
        }
        uint32_t o[kPerLane];
        uint32_t mine = 0;  // this lane's largest
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            o[i] = order_of(v[i]);
            mine = max(mine, o[i]);
        }
        float best = 0.0f, total = 0.0f;
        int got_id = -1;  // lane j keeps the token's j-th expert
        float got_w = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, mine);
            if (top == 0) break;
            unsigned at = 0xFFFFFFFFu;  // the lane's lowest expert with that logit
#pragma unroll
            for (int i = kPerLane - 1; i >= 0; --i)
                if (o[i] == top) at = i * 32 + lane;
            const int id = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, at));
            const float l = value_of(top);
            if (j == 0) {
                best = l;
                if (!a.renorm) {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i)
                        if (o[i]) s += expf(value_of(o[i]) - best);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
                    total = s;
                }
            }
            if (lane == j) {
                got_id = id;
                got_w = l;
            }
            mine = 0;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (i * 32 + lane == id) o[i] = 0;
                mine = max(mine, o[i]);
            }
        }
        // the weights of the k together
        float w = got_id >= 0 ? expf(got_w - best) : 0.0f;
        if (a.renorm) {
            total = w;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = got_id;
            a.weights[t * a.k + lane] = got_id < 0 ? 0.0f : w / total * a.scale;
            if (got_id >= 0) atomicAdd(&count[got_id], 1);
        }
    }
}

// Exclusive sums over the experts of `base` (its pairs), plus `prior` (those of
// earlier parts): the first row of an expert in this part; part 0 writes the
// offsets.  Returns all experts' rows.
__device__ __forceinline__ int32_t first_rows(int E, int32_t* base, const int32_t* prior, int32_t* offsets, int32_t* warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    int32_t rows = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        const int32_t n = e < E ? base[e] : 0;
        int32_t incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += u;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        const int32_t w = lane < warps ? warp_sums[lane] : 0;
        const int32_t below = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0);
        const int32_t all = __reduce_add_sync(0xFFFFFFFFu, w);
        const int32_t first = rows + below + incl - n;
        if (e < E) {
            base[e] = first + prior[e];
            if (offsets) offsets[e] = first;
        }
        rows += all;
        __syncthreads();
    }
    if (offsets && threadIdx.x == 0) offsets[E] = rows;
    return rows;
}

// The rows of the pairs of tokens first .. last - 1; `next` [kPlacers][E] is zero.
__device__ __forceinline__ void place(const Route& a, int64_t first, int64_t last, const int32_t* base, int32_t* next) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool placer = warp < kPlacers;
    int64_t w0 = 0, w1 = 0;
    if (placer) share(last - first, kPlacers, warp, &w0, &w1);
    const int64_t p0 = (first + w0) * a.k, p1 = (first + w1) * a.k;
    if (placer)
        for (int64_t p = p0 + lane; p < p1; p += 32) {
            const int e = a.ids[p];
            if (e >= 0) atomicAdd(&next[warp * a.E + e], 1);
        }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int32_t at = base[e];
#pragma unroll
        for (int w = 0; w < kPlacers; ++w) {
            const int32_t n = next[w * a.E + e];
            next[w * a.E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    if (placer)
        for (int64_t q = p0; q < p1; q += 32) {
            const int64_t p = q + lane;
            const int e = p < p1 ? a.ids[p] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
            int32_t row = -1;
            if (e >= 0) {
                row = next[warp * a.E + e] + __popc(same & ((1u << lane) - 1u));
                a.row_token[row] = static_cast<int32_t>(p / a.k);
            }
            __syncwarp();
            if (e >= 0 && lane == __ffs(same) - 1) next[warp * a.E + e] += __popc(same);
            __syncwarp();
            if (p < p1) a.token_row[p] = row;
        }
}

// row_token behind the last row
__device__ __forceinline__ void clear_rest(const Route& a, int32_t rows, int part, int parts) {
    for (int64_t r = rows + static_cast<int64_t>(part) * blockDim.x + threadIdx.x; r < a.T * a.k;
         r += static_cast<int64_t>(parts) * blockDim.x)
        a.row_token[r] = -1;
}

size_t shared_bytes(int E) { return sizeof(int32_t) * (kPlacers + 3) * E; }

// One cluster does all of it.
template <typename Logit, int kPerLane>
__global__ void __launch_bounds__(kThreadsOf<kPerLane>) route_cluster(const Route a) {
    extern __shared__ int32_t shared[];
    int32_t* count = shared;        // [E] of this part, read by all CTAs
    int32_t* base = count + a.E;    // [E] pairs of an expert, then its first row in this part
    int32_t* prior = base + a.E;    // [E] its pairs in earlier parts
    int32_t* next = prior + a.E;    // [kPlacers][E]
    __shared__ int32_t warp_sums[32];
    for (int i = threadIdx.x; i < (kPlacers + 3) * a.E; i += blockDim.x) shared[i] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    const int part = blockIdx.x, parts = gridDim.x;
    int64_t first, last;
    share(a.T, parts, part, &first, &last);
    choose<Logit, kPerLane>(a, first, last, count);
    if (parts > 1) cluster_sync_all();
    else __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int32_t all = 0, mine = 0;
        for (int c = 0; c < parts; ++c) {
            const int32_t n = c == part ? count[e] : ld_dsmem_s32(map_to_rank(smem_u32(count + e), c));
            all += n;
            if (c < part) mine += n;
        }
        base[e] = all;
        prior[e] = mine;
    }
    __syncthreads();
    if (parts > 1) cluster_arrive();  // (this CTA has read its peers' counts)
    const int32_t rows = first_rows(a.E, base, prior, part == 0 ? a.offsets : nullptr, warp_sums);
    place(a, first, last, base, next);
    clear_rest(a, rows, part, parts);
    if (parts > 1) cluster_wait();
}

template <typename Logit, int kPerLane>
__global__ void __launch_bounds__(kThreadsOf<kPerLane>) route_choose(const Route a) {
    __shared__ int32_t count[kPerLane * 32];
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    int64_t first, last;
    share(a.T, gridDim.x, blockIdx.x, &first, &last);
    choose<Logit, kPerLane>(a, first, last, count);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = count[e];
}

__global__ void __launch_bounds__(1024) route_place(const Route a) {
    extern __shared__ int32_t shared[];
    int32_t* base = shared;
    int32_t* prior = base + a.E;
    int32_t* next = prior + a.E;
    __shared__ int32_t warp_sums[32];
    for (int i = threadIdx.x; i < (kPlacers + 2) * a.E; i += blockDim.x) shared[i] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    const int part = blockIdx.x, parts = gridDim.x;
    // the parts' counts: a thread an expert, as many groups of threads as there are, each every
    // groups-th part (whole numbers: the order of the additions does not matter)
    const int groups = max(1, static_cast<int>(blockDim.x) / a.E);
    const int g = threadIdx.x / a.E;
    if (g < groups)
        for (int e = threadIdx.x - g * a.E; e < a.E; e += groups == 1 ? blockDim.x : a.E) {
            int32_t all = 0, mine = 0;
#pragma unroll 8
            for (int c = g; c < parts; c += groups) {
                const int32_t n = a.counts[static_cast<int64_t>(c) * a.E + e];
                all += n;
                if (c < part) mine += n;
            }
            atomicAdd(&base[e], all);
            atomicAdd(&prior[e], mine);
        }
    __syncthreads();
    const int32_t rows = first_rows(a.E, base, prior, part == 0 ? a.offsets : nullptr, warp_sums);
    int64_t first, last;
    share(a.T, parts, part, &first, &last);
    place(a, first, last, base, next);
    clear_rest(a, rows, part, parts);
}

cudaError_t launch(void (*kernel)(const Route), int grid, int threads, int cluster, size_t smem, cudaStream_t st,
                   const Route& r) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, r);
}

template <typename Logit, int kPerLane>
cudaError_t launch_sized(const Route& r, cudaStream_t st) {
    constexpr int kThreads = kThreadsOf<kPerLane>;
    if (r.T <= kClusterTokens) {  // a token a warp where one CTA has enough of them
        const int parts = r.T <= kThreads / 32 ? 1 : kClusterParts;
        return launch(route_cluster<Logit, kPerLane>, parts, kThreads, parts, shared_bytes(r.E), st, r);
    }
    const cudaError_t e = launch(route_choose<Logit, kPerLane>, kMaxParts, kThreads, 1, 0, st, r);
    return e != cudaSuccess ? e : launch(route_place, kMaxParts, 1024, 1, shared_bytes(r.E), st, r);
}

template <typename Logit>
cudaError_t launch_typed(const Route& r, cudaStream_t st) {
    if (r.E <= 32) return launch_sized<Logit, 1>(r, st);
    if (r.E <= 64) return launch_sized<Logit, 2>(r, st);
    if (r.E <= 128) return launch_sized<Logit, 4>(r, st);
    if (r.E <= 256) return launch_sized<Logit, 8>(r, st);
    if (r.E <= 512) return launch_sized<Logit, 16>(r, st);
    return launch_sized<Logit, 32>(r, st);
}

}  // namespace

size_t moe_route_workspace(int64_t T, int64_t E, int64_t k) {
    (void)k;
    return T <= kClusterTokens ? 0 : sizeof(int32_t) * static_cast<size_t>(E) * kMaxParts;
}

cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t st) {
    const Route r{a.logits, a.ld, a.T, a.E, a.k, a.renorm, a.scale, a.ids, a.weights, a.offsets, a.row_token,
                  a.token_row, a.workspace};
    return a.fp32 ? launch_typed<float>(r, st) : launch_typed<__nv_bfloat16>(r, st);
}

}  // namespace fp8k
