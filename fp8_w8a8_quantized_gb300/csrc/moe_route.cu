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
// in its own part, which some of the CTA's warps number 32 pairs at a time
// (match.sync).  Counts are whole numbers: nothing depends on an order of arrival.
//
// Up to some hundred tokens it is one launch of one cluster, whose CTAs read one
// another's counts through distributed shared memory; beyond, two launches with
// the counts in the workspace (choose, place).  Small calls are bound by latency
// (launch, logits, k rounds, numbering): 32 tokens of 64 experts, top 8, 5.1 us, of 128
// 5.5, 256 tokens of 128 6.7.  8192 tokens of 256 experts take 13.9 us (of 128 16.8) where
// their bytes take 1.4: two launches and their dependent reads 7, two tokens a warp 5, the
// numbering 2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr int kClusterParts = 8;
constexpr int kMaxParts = 152;  // of two launches: a CTA an SM

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

// items first .. last - 1 of n that are part `part`'s of `parts`
__device__ __forceinline__ void share(int n, int parts, int part, int* first, int* last) {
    const int per = n / parts, rem = n - per * parts;
    *first = part * per + min(part, rem);
    *last = *first + per + (part < rem ? 1 : 0);
}

// A lane's logits, largest first; of equal ones the lower expert first.  Up to 8
// they are sorted once (neighbours compared and exchanged, which keeps equal ones
// in order), so that taking one is a shift; with more, each round looks at all.
template <int N>
struct Lane {
    uint32_t o[N];
    uint32_t slots = 0;  // where o[0], o[1], ... come from, four bits each
    __device__ __forceinline__ explicit Lane(const uint32_t (&v)[N]) {
        static_assert(N <= 8, "");
        uint32_t at[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = v[i], at[i] = i;
#pragma unroll
        for (int r = 0; r < N; ++r)
#pragma unroll
            for (int i = r & 1; i + 1 < N; i += 2) {
                const bool turn = o[i] < o[i + 1];
                const uint32_t hi = max(o[i], o[i + 1]), lo = min(o[i], o[i + 1]);
                const uint32_t first = turn ? at[i + 1] : at[i], second = turn ? at[i] : at[i + 1];
                o[i] = hi, o[i + 1] = lo, at[i] = first, at[i + 1] = second;
            }
#pragma unroll
        for (int i = 0; i < N; ++i) slots |= at[i] << (4 * i);
    }
    __device__ __forceinline__ uint32_t head() const { return o[0]; }
    __device__ __forceinline__ uint32_t lowest() const { return slots & 15u; }
    __device__ __forceinline__ void pop(bool take) {
        if (!take) return;
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) o[i] = o[i + 1];
        o[N - 1] = 0;
        slots >>= 4;
    }
};

template <int N>
struct Wide {
    uint32_t o[N], top, at;
    __device__ __forceinline__ explicit Wide(const uint32_t (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = v[i];
        look();
    }
    __device__ __forceinline__ void look() {
        top = 0, at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (o[i] > top) top = o[i], at = i;
    }
    __device__ __forceinline__ uint32_t head() const { return top; }
    __device__ __forceinline__ uint32_t lowest() const { return at; }
    __device__ __forceinline__ void pop(bool take) {
        if (!take) return;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i == static_cast<int>(at)) o[i] = 0;
        look();
    }
};
template <>
struct Lane<16> : Wide<16> {
    using Wide<16>::Wide;
};
template <>
struct Lane<32> : Wide<32> {
    using Wide<32>::Wide;
};

struct Route {
    const void* logits;
    int64_t ld;
    int T, E, k;  // (T <= 2^23)
    bool renorm;
    float scale;
    int32_t* ids;
    float* weights;
    int32_t *offsets, *row_token, *token_row;
    uint16_t* counts;  // with two launches: [parts][E rounded up to 8]
};

// The experts of tokens first .. last - 1, counted in `count`.
template <typename Logit, int kPerLane>
__device__ __forceinline__ void choose(const Route& a, int first, int last, int32_t* count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Logit* logits = static_cast<const Logit*>(a.logits);
    constexpr int kWarps = kThreadsOf<kPerLane> / 32;
    float ahead[kPerLane];  // the warp's next token
    auto look = [&](int t) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = i * 32 + lane;
            ahead[i] = t < last && e < a.E ? logit(logits + static_cast<int64_t>(t) * a.ld + e) : -INFINITY;
        }
    };
    look(first + warp);
    for (int t = first + warp; t < last; t += kWarps) {
        float v[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) v[i] = ahead[i];
        look(t + kWarps);
        uint32_t o[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) o[i] = order_of(v[i]);
        float best = 0.0f, total = 0.0f;
        if (!a.renorm) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) m = o[i] ? fmaxf(m, v[i]) : m;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) total += o[i] ? expf(v[i] - m) : 0.0f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
        }
        Lane<kPerLane> mine(o);
        int got_id = -1;  // lane j keeps the token's j-th expert
        float got_w = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, mine.head());
            if (top == 0) break;
            const int id =
                static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, mine.head() == top ? mine.lowest() * 32 + lane : ~0u));
            if (j == 0) best = value_of(top);
            if (lane == j) {
                got_id = id;
                got_w = value_of(top);
            }
            mine.pop((id & 31) == lane);
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

// The rows of the pairs of tokens first .. last - 1; `next` [placers][E] is zero.
__device__ __forceinline__ void place(const Route& a, int first, int last, const int32_t* base, int32_t* next,
                                      int placers) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int w0 = 0, w1 = 0;
    if (warp < placers) share(last - first, placers, warp, &w0, &w1);
    const int p0 = (first + w0) * a.k, p1 = (first + w1) * a.k;
    int32_t* own = next + warp * a.E;
    int e = -1;         // of this lane's pair of the last 32, and which lanes have the same
    unsigned same = 0;
    auto take = [&](int q) {
        e = q + lane < p1 ? a.ids[q + lane] : -1;
        same = __match_any_sync(0xFFFFFFFFu, e);
    };
    auto count = [&] {
        if (e >= 0 && lane == __ffs(same) - 1) own[e] += __popc(same);
        __syncwarp();
    };
    for (int q = p0; q < p1; q += 32) {
        take(q);
        count();
    }
    __syncthreads();
    for (int x = threadIdx.x; x < a.E; x += blockDim.x) {
        int32_t at = base[x];
#pragma unroll 8
        for (int w = 0; w < placers; ++w) {
            const int32_t n = next[w * a.E + x];
            next[w * a.E + x] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int q = p0; q < p1; q += 32) {
        if (p1 - p0 > 32) take(q);
        int32_t row = -1;
        if (e >= 0) {
            row = own[e] + __popc(same & ((1u << lane) - 1u));
            a.row_token[row] = (q + lane) / a.k;
        }
        __syncwarp();
        count();
        if (q + lane < p1) a.token_row[q + lane] = row;
    }
}

// row_token behind the last row
__device__ __forceinline__ void clear_rest(const Route& a, int32_t rows, int part, int parts) {
    for (int64_t r = static_cast<int64_t>(rows) + part * static_cast<int>(blockDim.x) + threadIdx.x; r < a.T * a.k;
         r += parts * static_cast<int>(blockDim.x))
        a.row_token[r] = -1;
}

// (what 48 KB hold beside three numbers an expert)
int placers_of(int E) { return E <= 512 ? 16 : 8; }

size_t shared_bytes(int E) { return sizeof(int32_t) * (placers_of(E) * E + 3 * ((E + 7) & ~7)); }

// One cluster does all of it.
template <typename Logit, int kPerLane>
__global__ void __launch_bounds__(kThreadsOf<kPerLane>) route_cluster(const Route a, int placers) {
    extern __shared__ int32_t shared[];
    int32_t* count = shared;        // [E] of this part, read by all CTAs
    int32_t* base = count + a.E;    // [E] pairs of an expert, then its first row in this part
    int32_t* prior = base + a.E;    // [E] its pairs in earlier parts
    int32_t* next = prior + a.E;    // [placers][E]
    __shared__ int32_t warp_sums[32];
    for (int i = threadIdx.x; i < (placers + 3) * a.E; i += blockDim.x) shared[i] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    const int part = blockIdx.x, parts = gridDim.x;
    int first, last;
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
    place(a, first, last, base, next, placers);
    clear_rest(a, rows, part, parts);
    if (parts > 1) cluster_wait();
}

// Counts of a part lie in rows of E rounded up to 8, in 16 bits: every CTA of the second
// launch reads all of them, and a part has fewer than 2^16 tokens.
__host__ __device__ __forceinline__ int padded(int E) { return (E + 7) & ~7; }

template <typename Logit, int kPerLane>
__global__ void __launch_bounds__(kThreadsOf<kPerLane>) route_choose(const Route a, int) {
    __shared__ int32_t count[kPerLane * 32];
    for (int e = threadIdx.x; e < kPerLane * 32; e += blockDim.x) count[e] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    int first, last;
    share(a.T, gridDim.x, blockIdx.x, &first, &last);
    choose<Logit, kPerLane>(a, first, last, count);
    __syncthreads();
    for (int e = threadIdx.x; e < padded(a.E); e += blockDim.x) a.counts[blockIdx.x * padded(a.E) + e] = static_cast<uint16_t>(count[e]);
}

__global__ void __launch_bounds__(1024) route_place(const Route a, int placers) {
    extern __shared__ int32_t shared[];
    int32_t* base = shared;
    int32_t* prior = base + padded(a.E);
    int32_t* next = prior + padded(a.E);
    __shared__ int32_t warp_sums[32];
    for (int i = threadIdx.x; i < placers * a.E + 2 * padded(a.E); i += blockDim.x) shared[i] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    const int part = blockIdx.x, parts = gridDim.x;
    // the parts' counts: a thread eight experts of every groups-th part, all its loads on their way
    // together; a group is whole warps, so that lanes add to different numbers (whole ones: the
    // order does not matter)
    const int columns = padded(a.E) / 8, warps = (columns + 31) / 32;
    const int groups = min(16, static_cast<int>(blockDim.x) / 32 / warps);
    const int g = (threadIdx.x >> 5) / warps, x = threadIdx.x - g * warps * 32;
    if (g < groups && x < columns) {
        int32_t all[8] = {}, mine[8] = {};
        const uint4* counts = reinterpret_cast<const uint4*>(a.counts) + x;
#pragma unroll 10
        for (int c = g; c < parts; c += groups) {
            const uint4 n = counts[c * columns];
            const uint32_t w[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int32_t v = static_cast<int32_t>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
                all[i] += v;
                if (c < part) mine[i] += v;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (all[i]) atomicAdd(base + 8 * x + i, all[i]);
            if (mine[i]) atomicAdd(prior + 8 * x + i, mine[i]);
        }
    }
    __syncthreads();
    const int32_t rows = first_rows(a.E, base, prior, part == 0 ? a.offsets : nullptr, warp_sums);
    int first, last;
    share(a.T, parts, part, &first, &last);
    place(a, first, last, base, next, placers);
    clear_rest(a, rows, part, parts);
}

// One cluster up to here (top 2 to 8, cluster / two launches, us: 512 tokens of 8 experts 5.8 /
// 9.9, of 64 8.5 / 8.5, of 256 11.4 / 8.3).
int64_t cluster_tokens(int64_t E) { return E <= 64 ? 512 : E <= 256 ? 256 : 128; }

cudaError_t launch(void (*kernel)(const Route, int), int grid, int threads, int cluster, size_t smem, cudaStream_t st,
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
    return cudaLaunchKernelEx(&cfg, kernel, r, placers_of(r.E));
}

template <typename Logit, int kPerLane>
cudaError_t launch_sized(const Route& r, cudaStream_t st) {
    constexpr int kThreads = kThreadsOf<kPerLane>;
    if (r.T <= cluster_tokens(r.E)) {
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
    return T <= cluster_tokens(E) ? 0 : sizeof(uint16_t) * padded(static_cast<int>(E)) * kMaxParts;
}

cudaError_t launch_moe_route(const RouteArgs& a, cudaStream_t st) {
    const Route r{a.logits, a.ld, static_cast<int>(a.T), a.E, a.k, a.renorm, a.scale, a.ids, a.weights, a.offsets, a.row_token,
                  a.token_row, a.workspace};
    return a.fp32 ? launch_typed<float>(r, st) : launch_typed<__nv_bfloat16>(r, st);
}

}  // namespace fp8k
