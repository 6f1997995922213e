// Block tables, slot maps and positions of a serving step, built on the GPU
// from the requests' lengths.  With page size p, request b holds c_b cached
// tokens and brings n_b new ones:
//
//   have_b  = ceil(c_b / p),  need_b = ceil((c_b + n_b) / p)
//   first_b = sum_{a < b} (need_a - have_a),  cu_b = sum_{a < b} n_a
//   table[b, have_b + i] = free[first_b + i]              (i < need_b - have_b)
//   pos[cu_b + i] = c_b + i,  slot[cu_b + i] = table[b, pos / p] p + pos mod p
//
// There is next to nothing to compute: the call is bound by its launch and by
// two dependent global reads (the lengths, then the page of a token).  So it
// is ONE launch without a pass between the sums and their use: every CTA scans
// all the lengths itself (8 bytes a request out of L2) and then writes its own
// range of tokens and its share of the pages taken, a thread each, which finds
// its request by bisection in shared memory.  A token on a page that this very
// call takes looks the page up in `free`, not in the table, so no CTA reads
// what another one writes.  (Loads go past L1: the lines that this grid's start
// found there may be older than what the kernel before it wrote.)  Division by
// the page size is a multiplication (64-bit divisions alone took 6 of 11 us for
// 256 requests).
//
// Measured: 256 requests with a token each 3.1 us, 96 prompts of up to 1365
// tokens 4.8 us, back to back in a graph, where any launch takes 2.5 to 3.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr int kThreads = 256;

// x / d for x < 2^32: the high half of x ceil(2^64 / d) (d = 1: none fits, x).
struct Pages {
    uint64_t inverse;
    uint32_t size, width;
    __device__ uint32_t of(uint32_t x) const {
        return size == 1 ? x : static_cast<uint32_t>(__umul64hi(x, inverse));
    }
    // Pages of that many tokens, as far as a table row has room.
    __device__ uint32_t needed(uint32_t tokens) const {
        const uint32_t n = of(tokens);
        return min(n + (n * size < tokens ? 1u : 0u), width);
    }
};

struct Sums {
    int64_t tokens, pages;
};

// Inclusive block scan of one Sums per thread; `total` gets the block's sum.
__device__ __forceinline__ Sums scan_block(Sums v, Sums* warp_sums, Sums& total) {
    const int lane = lane_id(), warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v.tokens, o);
        const int64_t p = __shfl_up_sync(0xFFFFFFFFu, v.pages, o);
        if (lane >= o) {
            v.tokens += t;
            v.pages += p;
        }
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    total = Sums{0, 0};
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) {
            v.tokens += total.tokens;
            v.pages += total.pages;
        }
        total.tokens += warp_sums[w].tokens;
        total.pages += warp_sums[w].pages;
    }
    return v;
}

// The last of `starts[0 .. n]` (ascending) that is <= k.
__device__ __forceinline__ int find_start(const int64_t* starts, int n, int64_t k) {
    int a = 0, e = n;
    while (e - a > 1) {
        const int mid = (a + e) >> 1;
        if (starts[mid] <= k) a = mid; else e = mid;
    }
    return a;
}

// kPer: requests a thread; the lengths are scanned kThreads * kPer at a time.
template <int kPer>
__global__ void __launch_bounds__(kThreads)
    kv_slots(const int32_t* ctx, const int32_t* fresh, int64_t B, const int32_t* free_pages,
             int64_t n_free, const Pages page, int32_t* table, int64_t ld_table, int64_t T, int64_t per_cta,
             int64_t* __restrict__ slot, int32_t* __restrict__ pos, int32_t* __restrict__ cu,
             int32_t* __restrict__ lens, int32_t* __restrict__ used) {
    constexpr int kChunk = kThreads * kPer;
    __shared__ int64_t s_cu[kChunk + 1];     // first token of each request of the chunk
    __shared__ int64_t s_first[kChunk + 1];  // first page taken from `free`
    __shared__ uint32_t s_ctx[kChunk];
    __shared__ Sums warp_sums[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait_primary();

    const int64_t t_lo = blockIdx.x * per_cta;
    const int64_t t_hi = t_lo + per_cta < T ? t_lo + per_cta : T;
    Sums carry{0, 0};
    for (int64_t b0 = 0; b0 < B; b0 += kChunk) {
        const int n = static_cast<int>(B - b0 < kChunk ? B - b0 : kChunk);
        uint32_t c[kPer], f[kPer], take[kPer];
        Sums mine{0, 0};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = threadIdx.x * kPer + i;
            c[i] = r < n ? max(__ldcg(ctx + b0 + r), 0) : 0;
            f[i] = r < n ? max(__ldcg(fresh + b0 + r), 0) : 0;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            take[i] = page.needed(c[i] + f[i]) - page.needed(c[i]);  // (c + f < 2^32)
            mine.tokens += f[i];
            mine.pages += take[i];
        }
        Sums total;
        const Sums upto = scan_block(mine, warp_sums, total);
        int64_t t = carry.tokens + upto.tokens - mine.tokens;
        int64_t p = carry.pages + upto.pages - mine.pages;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = threadIdx.x * kPer + i;
            if (r < n) {
                s_cu[r] = t;
                s_first[r] = p;
                s_ctx[r] = c[i];
                if (blockIdx.x == 0) {
                    cu[b0 + r] = static_cast<int32_t>(t < T ? t : T);
                    lens[b0 + r] = static_cast<int32_t>(min(c[i] + f[i], 0x7FFFFFFFu));
                }
            }
            t += f[i];
            p += take[i];
        }
        carry.tokens += total.tokens;
        carry.pages += total.pages;
        if (threadIdx.x == 0) {
            s_cu[n] = carry.tokens;
            s_first[n] = carry.pages;
        }
        __syncthreads();

        // the pages that the requests take
        for (int64_t k = s_first[0] + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
             k < s_first[n]; k += static_cast<int64_t>(gridDim.x) * kThreads) {
            const int a = find_start(s_first, n, k);
            table[(b0 + a) * ld_table + page.needed(s_ctx[a]) + (k - s_first[a])] =
                k < n_free ? __ldcg(free_pages + k) : -1;
        }
        // this CTA's tokens that belong to the chunk's requests
        const int64_t lo = t_lo > s_cu[0] ? t_lo : s_cu[0];
        const int64_t hi = t_hi < s_cu[n] ? t_hi : s_cu[n];
        for (int64_t k = lo + threadIdx.x; k < hi; k += kThreads) {
            const int a = find_start(s_cu, n, k);
            const uint32_t at = s_ctx[a] + static_cast<uint32_t>(k - s_cu[a]);
            const uint32_t pg = page.of(at), have = page.needed(s_ctx[a]);
            int64_t id = -1;
            if (pg < have) {
                id = __ldcg(table + (b0 + a) * ld_table + pg);
            } else if (pg < page.width) {
                const int64_t i = s_first[a] + (pg - have);
                if (i < n_free) id = __ldcg(free_pages + i);
            }
            slot[k] = id < 0 ? -1 : id * page.size + (at - pg * page.size);
            pos[k] = static_cast<int32_t>(min(at, 0x7FFFFFFFu));
        }
        __syncthreads();
    }
    // room that no token needs
    for (int64_t k = (t_lo > carry.tokens ? t_lo : carry.tokens) + threadIdx.x; k < t_hi;
         k += kThreads) {
        slot[k] = -1;
        pos[k] = 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        cu[B] = static_cast<int32_t>(carry.tokens < T ? carry.tokens : T);
        *used = static_cast<int32_t>(carry.pages < INT32_MAX ? carry.pages : INT32_MAX);
    }
}

}  // namespace

cudaError_t launch_kv_slots(const int32_t* ctx, const int32_t* fresh, int64_t B,
                            const int32_t* free_pages, int64_t n_free, int64_t page,
                            int32_t* table, int64_t width, int64_t ld_table, int64_t T,
                            int64_t* slot, int32_t* pos, int32_t* cu, int32_t* lens,
                            int32_t* used, int num_sms, cudaStream_t st) {
    // a token a thread, as far as the SMs go
    const int64_t want = (T + kThreads - 1) / kThreads;
    const int64_t grid = want < 1 ? 1 : want < num_sms ? want : num_sms;
    Pages pages;
    pages.size = static_cast<uint32_t>(page);
    pages.width = static_cast<uint32_t>(width);
    pages.inverse = page == 1 ? 0 : ~uint64_t(0) / static_cast<uint64_t>(page) + 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (one request a thread costs the fewest requests the least; more of them
    // take fewer rounds of the scan with eight)
    return cudaLaunchKernelEx(&cfg, B <= kThreads ? kv_slots<1> : kv_slots<8>, ctx, fresh, B, free_pages,
                              n_free, pages, table, ld_table, T, (T + grid - 1) / grid, slot, pos, cu,
                              lens, used);
}

}  // namespace fp8k
