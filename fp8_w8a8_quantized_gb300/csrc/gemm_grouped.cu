// Products of each expert's rows with that expert's weights, rows sorted by
// expert with bounds known on the GPU alone:
//   a[r, n] = ((sum_k e4m3(xq[r, k]) e4m3(wq[e, n, k])) s_tok[r]) s_w[e, n]
//   y = bf16(a), or bf16(silu(a[:, n]) a[:, n + N / 2])
//
// One persistent launch: each worker counts every expert's tiles from the bounds
// and takes its share of the list.  A tile is 128 rows a CTA by 256 weight rows
// (with the gated activation 128 of the gate and the 128 of the values that go
// with them, so that both lie in the same lanes of tensor memory).  Rows are on
// the MMA's M side even where an expert has few: the weights are then read as
// fast as DRAM gives them with the tensor cores a third busy, and the rows that
// an expert does not have cost next to no loads (a box of 32, 64 or 128 rows) and
// no stores.  What MMAs read there is whatever the ring held; it reaches outputs of
// those rows alone, which nothing reads.
//   kPair = false: a worker is a CTA (cta_group::1).  For few rows an expert: an
//     SM alone streams weights of its own, and there are twice as many workers.
//   kPair = true: a worker is two CTAs on two SMs (cta_group::2, 256 x 256 tiles):
//     half the loads into shared memory per product.  An expert's last rows, 128
//     at most, take a tile of M = 128.
//
// The list: tile t of an expert's ceil(rows / tile rows) x ceil(N / 256), row
// tiles next to one another, so that workers that run at the same time share
// weights in L2.  Workers take whole tiles in turn; the tiles of the last,
// unfull round are cut along K where that is sooner done (grouped_plan.h).  A
// worker that has part of a tile leaves its sums in the workspace, and the last of
// a tile's workers to arrive (a counter, zeroed by the kernel before) adds the
// parts in the order of K: the order of every sum is fixed by the sizes and
// bounds.  No worker waits for another.
//
// Per CTA 320 threads: warp 0 loads (TMA; stages of 128 of K, as more and smaller
// ones keep more of the ring on its way: 8 x 1024 rows 619 us with 256 a stage, 547
// with 128), warp 1 issues the MMAs (in a pair the even CTA's), warps 2 to 9 scale,
// round and store.  Both issuing warps wait as a whole and issue from uniform
// registers (547 -> 491 us).
//
// Measured: 8 x 8 rows of 4096 x 28672 136 us, 6.9 TB/s of weights (102% of a
// copy); 64 x 32 rows of 2048 x 2816 59 us, 6.4 TB/s; 4096 tokens on two of eight
// experts 585 us, 3.3 PFLOP/s with the tensor cores 89% busy at the 1.6 GHz that the
// card's power leaves.  40 experts of 0 to 2866 rows, 1408 x 2048: 57 us where bytes
// take 31: between tiles of only 11 stages 1.3 of 4.9 us go to the outputs' way to
// memory and the accumulators' hand-over, and 13% of the tiles' rows are empty (25%
// where a tile of 128 rows counts as one of 256).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "grouped_plan.h"
#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

using grouped::Bounds;
using grouped::Costs;
using grouped::Walk;

constexpr int kOutWarps = 8;      // two for each 32 rows of a CTA's tile
constexpr int kThreads = 64 + 32 * kOutWarps;
constexpr int kTileRows = 128;    // rows a CTA
constexpr int BN = 256;           // accumulator columns
constexpr int kHalf = 128;        // weight rows of a TMA box (of a small tile's: kHalf / 2)
constexpr int kMinBox = 32;       // rows of X of the smallest of three TMA boxes (32, 64, 128)
constexpr int BK = 128;           // K of a stage: one swizzled column of 128 bytes
constexpr int KSTEP = 32;         // K of one tcgen05.mma kind::f8f6f4
constexpr int kAccBufs = 2;
constexpr uint32_t TMEM_COLS = kAccBufs * BN;
constexpr int kMaxExperts = 1024;
constexpr int kMaxCtas = 152;
constexpr int kBatch = 4;         // rows whose parts are added at a time
constexpr int kPrefetched = 8;    // stages whose weights are asked for ahead of the start

template <bool kPair>
struct Cfg {
    static constexpr int CTAS = kPair ? 2 : 1;
    static constexpr int BM = kTileRows * CTAS;
    static constexpr int STAGES = kPair ? 6 : 4;
    static constexpr int B_ROWS = BN / CTAS;      // weight rows in this CTA
    static constexpr uint32_t A_TILE = kTileRows * BK;
    static constexpr uint32_t B_TILE = B_ROWS * BK;
    static constexpr uint32_t RING = STAGES * (A_TILE + B_TILE);
};

template <int kStages>
struct Bars {
    uint64_t full[kStages];    // pair: the even CTA's
    uint64_t empty[kStages];
    uint64_t acc_full[kAccBufs];
    uint64_t acc_empty[kAccBufs];  // pair: the even CTA's
    uint64_t drain;
    uint64_t part_done;            // the epilogue warps have written their part of a tile
    uint64_t verdict;              // `last` is set
    uint32_t tmem_base;
    int abort;
    int last;                      // this CTA is the last of the tile's to arrive
    alignas(16) float s_w[kOutWarps][BN / 2];     // weight scales of the warp's columns
    alignas(16) uint4 out[kOutWarps][32 * 4];     // 32 rows x 64 bytes on their way out
    int first[kMaxExperts + 1];    // tiles of the experts below
    int begin[kMaxExperts], end[kMaxExperts];  // an expert's rows
};

template <bool kPair>
constexpr size_t smem_bytes() {
    return 1024 + Cfg<kPair>::RING + sizeof(Bars<Cfg<kPair>::STAGES>);
}

struct Args {
    const float* s_tok;
    const float* s_w;
    const int32_t* offsets;
    __nv_bfloat16* y;
    unsigned* count;   // [workers][CTAS]
    float* parts;      // [workers][CTAS][2][slot]
    int64_t slot;      // floats of a part: its rows x BN
    int E, R, N, K;
    Costs costs;
    unsigned* status;
};

// X in boxes of 32, 64 and 128 rows, W in boxes of kHalf and kHalf / 2 rows.
struct Maps {
    CUtensorMap x[3], w, w_small;
};

// (from L2: read before the wait and again behind it)
__device__ __forceinline__ Bounds bounds_of(const Args& a, int e) {
    return grouped::bounds_within(__ldcg(a.offsets + e), __ldcg(a.offsets + e + 1), a.R);
}

// Where a tile lies.
struct Place {
    int e, row0, rows, n_blk;  // its first row, how many rows the expert has from there on
};
template <typename B, int BM>
struct Finder {
    const B* bars;
    int experts, e = -1, m_tiles = 1;
    __device__ __forceinline__ Place at(int tile) {
        const int* first = bars->first;
        if (e < 0 || tile < first[e] || tile >= first[e + 1]) {
            int lo = 0, hi = experts;  // first[lo] <= tile < first[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= tile) lo = mid;
                else hi = mid;
            }
            e = lo;
            m_tiles = (bars->end[e] - bars->begin[e] + BM - 1) / BM;
        }
        const int local = tile - first[e];
        const int n = local / m_tiles, m = local - n * m_tiles;
        return {e, bars->begin[e] + m * BM, bars->end[e] - bars->begin[e] - m * BM, n};
    }
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool kPair, bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ Maps maps, const Args a) {
    using C = Cfg<kPair>;
    using B = Bars<C::STAGES>;
    constexpr int kOut = kGated ? BN / 2 : BN;  // outputs of a tile's row
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    uint8_t* sA = smem;
    uint8_t* sB = smem + C::STAGES * C::A_TILE;
    B* bars = reinterpret_cast<B*>(smem + C::RING);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
    const bool leader = rank == 0;
    const int worker = blockIdx.x / C::CTAS, workers = gridDim.x / C::CTAS;
    const int F = kGated ? a.N / 2 : a.N;
    const int nk = (a.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int b = 0; b < kAccBufs; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], kOutWarps * C::CTAS);
        }
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->part_done, kOutWarps);
        mbar_init(&bars->verdict, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < 3; ++i) tma_prefetch_desc(&maps.x[i]);
        tma_prefetch_desc(&maps.w);
        if constexpr (kPair) tma_prefetch_desc(&maps.w_small);
    }
    if (warp == 1) tmem_take<kPair>(&bars->tmem_base, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    pdl_launch_dependents();  // (behind the allocation: see ptx.cuh)
    if constexpr (kPair) cluster_sync_all();  // the peer's barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    volatile int* abort_flag = &bars->abort;

    // tiles of each expert, then of all below it
    const int n_tiles = (F + kOut - 1) / kOut;
    auto make_list = [&] {
        auto tiles_of = [&](int rows) { return (rows + C::BM - 1) / C::BM * n_tiles; };
        bool back = false;
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            const Bounds b = bounds_of(a, e);
            bars->begin[e] = b.begin, bars->end[e] = b.end;
            bars->first[e + 1] = tiles_of(b.end - b.begin);
            back |= b.back;
        }
        if (__syncthreads_or(back)) {  // (bounds that no routing makes)
            if (threadIdx.x == 0) {
                grouped::put_in_order(bars->begin, bars->end, a.E);
                for (int e = 0; e < a.E; ++e) bars->first[e + 1] = tiles_of(bars->end[e] - bars->begin[e]);
            }
            __syncthreads();
        }
        if (warp == 0) {
            int sum = 0;
            for (int e0 = 0; e0 < a.E; e0 += 32) {
                int v = e0 + lane < a.E ? bars->first[e0 + lane + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
                    if (lane >= d) v += u;
                }
                if (e0 + lane < a.E) bars->first[e0 + lane + 1] = sum + v;
                sum += __shfl_sync(0xFFFFFFFFu, v, 31);
            }
            if (lane == 0) bars->first[0] = 0;
        }
        __syncthreads();
    };
    // The kernel before (the quantizer, or the one that clears the counters) lets this one start when
    // all work before it is done, so that the bounds are there already: the list is made and the
    // weights of the first stages are brought into L2 while it runs.  Behind the wait the bounds are
    // read again, and the list made again if they are others.  (Against a start beside the work before
    // that kernel, in a graph: 1 token on two of eight experts 44.0 -> 42.1 us, 16 tokens 121.7 -> 117.5,
    // 32 tokens 139.3 -> 134.3, 253 tokens on 8 of 64 60.9 -> 60.3.)
    make_list();
    if (warp == 0) {
        Walk first(bars->first[a.E], workers, worker, nk, a.costs);
        if (first.advance()) {
            const Place p = Finder<B, C::BM>{bars, a.E}.at(first.tile);
            const int n0 = p.n_blk * kOut;
            const int w_first = p.e * a.N + n0, w_second = w_first + (kGated ? F : kHalf);
            const int stages = min(first.kb1 - first.kb0, kPrefetched);
            if (lane < 2 * stages && (kGated || n0 + (lane & 1) * kHalf < F) && (!kPair || (lane & 1) == rank))
                tma_prefetch_l2_2d(&maps.w, (first.kb0 + (lane >> 1)) * BK, lane & 1 ? w_second : w_first);
        }
        __syncwarp();
    }
    pdl_wait_primary();
    bool same = true;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const Bounds b = bounds_of(a, e);
        same = same && b.begin == bars->begin[e] && b.end == bars->end[e];
    }
    if (!__syncthreads_and(same)) make_list();
    Walk walk(bars->first[a.E], workers, worker, nk, a.costs);
    Finder<B, C::BM> find{bars, a.E};

    if (warp == 0) {
        // ---- loads: this CTA's rows of X, its part of the weight rows ----
        uint32_t stage = 0, phase = 0, issued = 0;
        const uint64_t once = policy_evict_first(), again = policy_evict_normal();
        bool ok = true;
        while (ok && walk.advance()) {
            const Place p = find.at(walk.tile);
            const bool small = kPair && p.rows <= kTileRows;
            const int cta_rows = small ? kTileRows / 2 : kTileRows;
            // rows of X in one box, the smallest that has them (further rows of it are another
            // expert's: a copy costs the loading warp more than they cost)
            auto box_of = [&](int cta) {  // 0: no rows
                const int rows = min(p.rows - cta * cta_rows, cta_rows);
                return rows <= 0 ? 0 : rows <= kMinBox ? kMinBox : rows <= 2 * kMinBox ? 2 * kMinBox : 4 * kMinBox;
            };
            const int box = box_of(rank);
            const CUtensorMap* x_map = maps.x + (box >> 6);  // 32, 64, 128 -> 0, 1, 2
            const int row = p.row0 + rank * cta_rows;
            // weight rows, halves of the tile's columns: with a gate the gate's and the values' (in a
            // small tile both CTAs have 64 of each), or 128 and 128.  A half that is beyond the
            // expert's rows is left out.
            const int n0 = p.n_blk * kOut;
            const int w_first = p.e * a.N + n0, w_second = w_first + (kGated ? F : kHalf);
            const bool second = kGated || n0 + kHalf < F;
            const bool quarters = kGated && small;
            const int w_row = quarters ? w_first + rank * (kHalf / 2) : rank ? w_second : w_first;
            const bool w_there = rank == 0 || second;
            // of K, that the stage's barrier waits for
            const uint32_t bytes = (kPair ? box_of(0) + box_of(1) : box) + (second ? 2 : 1) * kHalf;
            // weights that one row tile reads leave L2 first, to what is read again (8 x 8 rows 141 ->
            // 136 us; where several do, 570 -> 604)
            const uint64_t policy = find.m_tiles == 1 ? once : again;
            // (operands of the copies from uniform registers, see elect_one in ptx.cuh)
            const uint32_t tx = uniform(bytes) * BK;
            const int x_row = static_cast<int>(uniform(row));
            const int w_row0 = static_cast<int>(uniform(kPair ? w_row : w_first)), w_row1 = static_cast<int>(uniform(kPair ? w_row + F : w_second));
            const bool has_x = uniform(box) != 0, has_w = uniform(w_there), both = uniform(kPair ? quarters : second);
            for (int kb = walk.kb0; kb < walk.kb1; ++kb) {
                if (!(ok = warp_ready(&bars->empty[stage], phase ^ 1u, abort_flag, a.status))) break;
                if (elect_one()) {
                    uint8_t* w = sB + stage * C::B_TILE;
                    const int k = kb * BK;
                    uint64_t* full = &bars->full[stage];
                    const uint32_t full0 = kPair ? map_to_rank(smem_u32(full), 0) : 0u;
                    auto load_w = [&](uint8_t* to, const CUtensorMap* map, int r) {
                        if constexpr (kPair) tma_load_2d_pair_hint(to, map, full0, k, r, policy);
                        else tma_load_2d_hint(to, map, full, k, r, policy);
                    };
                    if (leader) mbar_arrive_expect_tx(full, tx);
                    if constexpr (kPair) {
                        if (kGated && both) {
                            load_w(w, &maps.w_small, w_row0);
                            load_w(w + (kHalf / 2) * BK, &maps.w_small, w_row1);
                        } else if (has_w) {
                            load_w(w, &maps.w, w_row0);
                        }
                    } else {
                        load_w(w, &maps.w, w_row0);
                        if (both) load_w(w + kHalf * BK, &maps.w, w_row1);
                    }
                    if (has_x) {
                        uint8_t* x = sA + stage * C::A_TILE;
                        if constexpr (kPair) tma_load_2d_pair(x, x_map, full0, k, x_row);
                        else tma_load_2d(x, x_map, full, k, x_row);
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && leader && lane == 0) {  // copies in flight land before the shared memory goes away
            for (uint32_t j = issued > C::STAGES ? issued - C::STAGES : 0; j < issued; ++j)
                wait_landed(&bars->full[j % C::STAGES], (j / C::STAGES) & 1u, a.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            // ---- MMAs ----
            // (the next piece is looked up while the present one's MMAs run)
            uint32_t stage = 0, phase = 0;
            int local = 0;
            auto shape = [&] {
                return uniform(kPair && find.at(walk.tile).rows <= kTileRows ? idesc_e4m3_f32(kTileRows, BN)
                                                                             : idesc_e4m3_f32(C::BM, BN));
            };
            bool ok = true, more = walk.advance();
            uint32_t next_idesc = more ? shape() : 0u;
            while (ok && more) {
                const int kb0 = walk.kb0, kb1 = walk.kb1;
                const uint32_t idesc = next_idesc;
                const int buf = local % kAccBufs;
                const uint32_t acc_phase = (local / kAccBufs) & 1;
                ++local;
                if (!(ok = warp_wait_cluster(&bars->acc_empty[buf], acc_phase ^ 1u, abort_flag, a.status))) break;
                tc_fence_after();
                const uint32_t d = uniform(tmem_base + buf * BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = warp_ready(&bars->full[stage], phase, abort_flag, a.status))) break;
                    tc_fence_after();
                    const uint32_t xa = uniform(smem_u32(sA + stage * C::A_TILE));
                    const uint32_t wb = uniform(smem_u32(sB + stage * C::B_TILE));
                    const uint32_t add = uniform(kb != kb0);
                    const int steps = (a.K - kb * BK + KSTEP - 1) / KSTEP;  // (the last stage may have fewer)
                    if (elect_one()) {
                        const uint64_t a0 = sdesc_kmajor_sw128(xa), b0 = sdesc_kmajor_sw128(wb);
                        auto mma = [&](int kk) {
                            const uint64_t ad = a0 + 2 * kk, bd = b0 + 2 * kk;
                            if constexpr (kPair) mma_f8_pair(d, ad, bd, idesc, kk ? 1u : add);
                            else mma_f8(d, ad, bd, idesc, kk ? 1u : add);
                        };
                        if (steps >= BK / KSTEP) {
#pragma unroll
                            for (int kk = 0; kk < BK / KSTEP; ++kk) mma(kk);
                        } else {
                            for (int kk = 0; kk < steps; ++kk) mma(kk);
                        }
                        if constexpr (kPair) mma_commit_pair(&bars->empty[stage], 0x3);
                        else mma_commit(&bars->empty[stage]);
                    }
                    __syncwarp();
                    if (kb == kb0) {
                        more = walk.advance();
                        if (more) next_idesc = shape();
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok && elect_one()) {
                    if constexpr (kPair) mma_commit_pair(&bars->acc_full[buf], 0x3);
                    else mma_commit(&bars->acc_full[buf]);
                }
                __syncwarp();
            }
            // every MMA has finished before tensor memory is freed
            if (elect_one()) {
                if constexpr (kPair) mma_commit_pair(&bars->drain, 0x1);
                else mma_commit(&bars->drain);
                wait_drain(&bars->drain, a.status);
            }
            __syncwarp();
        }
    } else {
        // ---- outputs: a warp has 32 of this CTA's 128 rows and half of the columns ----
        const int me = warp - 2, quarter = warp & 3, half = me >> 2;
        float* sw = bars->s_w[me];
        uint4* stage = bars->out[me];
        const bool wide = F % 8 == 0;  // rows of y at 16-byte boundaries
        int local = 0;
        uint32_t part_phase = 0;
        // a piece of the list as this warp sees it
        struct Piece {
            Place p;
            int tile, kb0, kb1;
            int cta_row0, first_row;  // the CTA's and the warp's first row within the tile
            int column0, chunks;      // outputs in chunks of 32: the warp's first and how many
            bool small;
            float st, sw[4];          // scales of the lane's row, of the warp's columns (128: 4 a lane)
        };
        // Its scales are asked for while the piece before is on its way out.
        auto look = [&](Piece& q) {
            q.p = find.at(walk.tile);
            q.tile = walk.tile, q.kb0 = walk.kb0, q.kb1 = walk.kb1;
            // A small tile (M = 128 over the pair): 64 rows a CTA, lanes 0 .. 63 with the first half
            // of the columns, lanes 64 .. 127 with the second.
            q.small = kPair && q.p.rows <= kTileRows;
            q.cta_row0 = rank * (q.small ? kTileRows / 2 : kTileRows);
            q.first_row = q.cta_row0 + (q.small ? quarter & 1 : quarter) * 32;
            q.chunks = (q.small ? kOut / 2 : kOut) / 64;
            q.column0 = (q.small ? (quarter >> 1) * (kOut / 2) : 0) + 32 * half * q.chunks;
            if (q.first_row >= q.p.rows) return;
            if (q.first_row + lane < q.p.rows) q.st = a.s_tok[q.p.row0 + q.first_row + lane];
            const float* s_w = a.s_w + static_cast<int64_t>(q.p.e) * a.N;
            const int n_first = q.p.n_blk * kOut + q.column0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = i * 32 + lane;  // (with a gate: 64 of the gate, 64 of the values)
                const int n = n_first + (kGated ? c & 63 : c);
                q.sw[i] = n < F ? s_w[n + (kGated && c >= 64 ? F : 0)] : 0.0f;
            }
        };
        Piece next = {};
        bool more = walk.advance();
        if (more) look(next);
        while (more) {
            const Piece now = next;
            const Place& p = now.p;
            const bool small = now.small;
            const int buf = local % kAccBufs;
            const uint32_t acc_phase = (local / kAccBufs) & 1;
            ++local;
            const int cta_row0 = now.cta_row0, first_row = now.first_row;
            const int cta_rows = min(p.rows - cta_row0, small ? kTileRows / 2 : kTileRows);
            const int here = min(32, p.rows - first_row);
            const bool any = here > 0, whole = now.kb0 == 0 && now.kb1 == nk;
            const bool row_ok = lane < here;
            const int64_t row = static_cast<int64_t>(p.row0) + first_row + lane;
            const int n0 = p.n_blk * kOut, n_first = n0 + now.column0;
            const int column0 = now.column0 - 32 * half * now.chunks;  // of the lanes
            const int chunks = now.chunks, chunk0 = half * chunks;
            const int up = small ? kOut / 2 : kOut;  // columns from a gate to its value in tensor memory
            const float st = row_ok ? now.st : 0.0f;
            if (any && whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sw[i * 32 + lane] = now.sw[i];
                __syncwarp();
            }
            more = walk.advance();
            if (more) look(next);
            // Rows at 16-byte boundaries go through shared memory, so that a store instruction writes
            // 64 bytes of eight rows each instead of 16 bytes of 32 rows: this lane's j-th piece of
            // 16 bytes of 4 (turned by the row: no bank is met twice), ...
            auto piece = [&](int j) -> uint4& { return stage[lane * 4 + (j ^ ((lane >> 1) & 3))]; };
            // ... and the pieces to rows at `out`, `row_bytes` apart, of which `bytes` are left.
            auto flush = [&](void* out, int64_t row_bytes, int64_t bytes) {
                __syncwarp();
                uint8_t* to = static_cast<uint8_t*>(out) + (lane >> 2) * row_bytes + 16 * (lane & 3);
                const bool there = 16 * (lane & 3) < bytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * i + (lane >> 2);
                    if (r < here && there)
                        __stcg(reinterpret_cast<uint4*>(to + 8 * i * row_bytes),
                               stage[r * 4 + ((lane & 3) ^ ((r >> 1) & 3))]);
                }
                __syncwarp();
            };
            // 32 outputs of this lane's row, the warp's i-th chunk
            auto emit = [&](const float (&v)[32], int i) {
                uint32_t packed[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                const int n = n_first + 32 * i;
                if (wide) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        piece(j) = make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                    flush(a.y + (static_cast<int64_t>(p.row0) + first_row) * F + n, 2 * static_cast<int64_t>(F),
                          2 * (static_cast<int64_t>(F) - n));
                    return;
                }
                if (!row_ok) return;
                // (unrolled with a guard a column, so that packed[] stays in registers)
                uint16_t* o = reinterpret_cast<uint16_t*>(a.y + row * F + n);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (n + j < F) o[j] = static_cast<uint16_t>(packed[j >> 1] >> ((j & 1) * 16));
            };
            // (acc s_tok) s_w of 32 columns, a pair of values an instruction
            auto scale = [&](float (&v)[32], const uint32_t (&r)[32], const float* w) {
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    mul2(v[j], v[j + 1], __uint_as_float(r[j]), __uint_as_float(r[j + 1]), st, st);
                    mul2(v[j], v[j + 1], v[j], v[j + 1], w[j], w[j + 1]);
                }
            };
            // g / (1 + exp(-g)) u, by exp(-|g|), so that the divisor lies in 1 .. 2.  (A quotient that
            // is rounded to 2^-22 and takes the same time for every value: rows that are not there
            // hold anything, and a true division of NaN takes 50 times as long.)
            auto gated = [&](float g, float u) {
                const float t = __expf(-fabsf(g));
                return __fdividef(g >= 0.0f ? g : g * t, 1.0f + t) * u;
            };
            auto release = [&] {  // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (kPair) mbar_arrive_cluster(map_to_rank(smem_u32(&bars->acc_empty[buf]), 0));
                    else mbar_arrive(&bars->acc_empty[buf]);
                }
            };
            if (!warp_wait(&bars->acc_full[buf], acc_phase, abort_flag, a.status)) break;
            tc_fence_after();
            const uint32_t acc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + buf * BN;
            if (cta_rows <= 0 || (whole && !any)) {
                release();
                continue;
            }
            if (whole) {
                const uint32_t from = acc + 32 * chunk0;
                if constexpr (kGated) {
#pragma unroll
                    for (int c = 0; c < kOut / 64; ++c) {
                        if (c >= chunks) break;
                        uint32_t g[32], u[32];
                        tmem_ld_32x32b_x32(from + 32 * c, g);
                        tmem_ld_32x32b_x32(from + up + 32 * c, u);
                        tmem_ld_wait_regs(g);
                        tmem_ld_wait_regs(u);
                        if (c == chunks - 1) release();
                        float v[32], x[32];
                        scale(v, g, sw + 32 * c);
                        scale(x, u, sw + 64 + 32 * c);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = gated(v[j], x[j]);
                        emit(v, c);
                    }
                } else {
                    // (chunk c + 1 is on its way while chunk c is scaled and stored)
                    uint32_t ra[32], rb[32];
                    auto one = [&](const uint32_t (&r)[32], int c) {
                        float v[32];
                        scale(v, r, sw + 32 * c);
                        emit(v, c);
                    };
                    tmem_ld_32x32b_x32(from, ra);
                    tmem_ld_wait_regs(ra);
#pragma unroll
                    for (int c = 0; c < kOut / 64; c += 2) {
                        if (c >= chunks) break;
                        tmem_ld_32x32b_x32(from + (c + 1) * 32, rb);
                        one(ra, c);
                        tmem_ld_wait_regs(rb);
                        if (c + 2 < chunks) tmem_ld_32x32b_x32(from + (c + 2) * 32, ra);
                        else release();
                        one(rb, c + 1);
                        if (c + 2 < chunks) tmem_ld_wait_regs(ra);
                    }
                }
                __syncwarp();
                continue;
            }
            // Part of a tile: the sums go to the workspace, row by row, this warp's half of the
            // lanes' chunks.
            auto part = [&](int w, int slot) {
                return a.parts + ((static_cast<int64_t>(w) * C::CTAS + rank) * 2 + slot) * a.slot;
            };
            if (any) {
                float* mine = part(worker, now.kb0 == 0 ? 1 : 0) + (first_row - cta_row0) * BN;
#pragma unroll
                for (int i = 0; i < BN / 64; ++i) {
                    const int mine_of = (small ? BN / 2 : BN) / 64;
                    if (i >= mine_of) break;
                    const int c = half * mine_of + i;
                    // (columns as in a tile of all rows: the gate's, then the values')
                    const int column = !small ? 32 * c
                                       : kGated ? column0 + 32 * (c & 1) + (c >> 1) * kOut
                                                : column0 + 32 * c;
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(acc + 32 * c, r);
                    tmem_ld_wait_regs(r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            piece(j) = make_uint4(r[16 * h + 4 * j], r[16 * h + 4 * j + 1], r[16 * h + 4 * j + 2],
                                                  r[16 * h + 4 * j + 3]);
                        flush(mine + column + 16 * h, BN * 4, 64);
                    }
                }
            }
            release();
            const int64_t unit = static_cast<int64_t>(now.tile - walk.whole) * nk;
            const int w_first = walk.worker_of(unit), w_last = walk.worker_of(unit + nk - 1);
            __threadfence();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->part_done);
            if (me == 0) {
                if (!warp_wait(&bars->part_done, part_phase, abort_flag, a.status)) break;
                if (lane == 0) {
                    __threadfence();
                    const unsigned before = atomicAdd(a.count + w_first * C::CTAS + rank, 1u);
                    bars->last = before == static_cast<unsigned>(w_last - w_first);
                    mbar_arrive(&bars->verdict);
                }
                __syncwarp();
            }
            if (!warp_wait(&bars->verdict, part_phase, abort_flag, a.status)) break;
            __syncwarp();
            part_phase ^= 1u;
            if (!*const_cast<volatile int*>(&bars->last)) continue;
            __threadfence();
            // The last to arrive adds the parts in the order of K: the warps take kBatch rows in turn,
            // a lane columns 4 l .. 4 l + 3 of each half (with a gate: the gate and its values).
            const int64_t step = a.slot * 2 * C::CTAS;
            float sl[4], sh[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + 4 * lane + j, m = kGated ? n : n + BN / 2;
                const float* s_w = a.s_w + static_cast<int64_t>(p.e) * a.N;
                sl[j] = n < F ? s_w[n] : 0.0f;
                sh[j] = m < F ? s_w[m + (kGated ? F : 0)] : 0.0f;
            }
            auto put = [&](const float (&q)[4], int r, int n) {
                __nv_bfloat16* out = a.y + (static_cast<int64_t>(p.row0) + cta_row0 + r) * F + n;
                if (wide) {
                    if (n < F)
                        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(q[0], q[1]), pack_bf16x2(q[2], q[3]));
                    return;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < F) out[j] = __float2bfloat16_rn(q[j]);
            };
            for (int r0 = me * kBatch; r0 < cta_rows; r0 += kOutWarps * kBatch) {
                float4 lo[kBatch], hi[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) lo[i] = hi[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const float* from = part(w_first, 1) + r0 * BN + 4 * lane;
                for (int w = w_first; w <= w_last; ++w) {
                    float4 l[kBatch], h[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (r0 + i < cta_rows) {
                            l[i] = __ldcg(reinterpret_cast<const float4*>(from + i * BN));
                            h[i] = __ldcg(reinterpret_cast<const float4*>(from + i * BN + BN / 2));
                        }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (r0 + i < cta_rows) {
                            lo[i].x += l[i].x, lo[i].y += l[i].y, lo[i].z += l[i].z, lo[i].w += l[i].w;
                            hi[i].x += h[i].x, hi[i].y += h[i].y, hi[i].z += h[i].z, hi[i].w += h[i].w;
                        }
                    from = w == w_first ? part(w_first + 1, 0) + r0 * BN + 4 * lane : from + step;
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (r0 + i >= cta_rows) break;
                    const float t = a.s_tok[p.row0 + cta_row0 + r0 + i];
                    float v[4] = {(lo[i].x * t) * sl[0], (lo[i].y * t) * sl[1], (lo[i].z * t) * sl[2], (lo[i].w * t) * sl[3]};
                    float u[4] = {(hi[i].x * t) * sh[0], (hi[i].y * t) * sh[1], (hi[i].z * t) * sh[2], (hi[i].w * t) * sh[3]};
                    if constexpr (kGated) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = gated(v[j], u[j]);
                        put(v, r0 + i, n0 + 4 * lane);
                    } else {
                        put(v, r0 + i, n0 + 4 * lane);
                        put(u, r0 + i, n0 + BN / 2 + 4 * lane);
                    }
                }
            }
            __syncwarp();
        }
    }

    // Neither CTA of a pair may free tensor memory or exit while MMAs, the peer's
    // copies or its arrivals can still touch it.
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_give_back<kPair>(tmem_base, TMEM_COLS);
    }
}

__global__ void clear_counts(unsigned* count, int n) {
    pdl_wait_primary();
    pdl_launch_dependents();  // (behind the wait: the products read the bounds ahead of theirs)
    for (int i = threadIdx.x; i < n; i += blockDim.x) count[i] = 0;
}

constexpr int64_t kCounts = kMaxCtas;
constexpr int64_t kCountBytes = (kCounts * 4 + 255) / 256 * 256;

// Floats of a part: the rows that a CTA can have, in 32s.
int64_t slot_floats(int64_t R) {
    const int64_t rows = (R + 31) / 32 * 32;
    return (rows < kTileRows ? rows : kTileRows) * BN;
}

// Pairs where an expert has more rows than a CTA's tile on average (2048 x 2816, rows an expert,
// single / pairs, us: 32 63.4 / 64.7, 128 67.2 / 69.2, 160 81.5 / 73.8; 14336 x 4096, 40 rows 77.7 /
// 89.9: half as many workers for as many tiles).
bool pairs_of(int64_t E, int64_t R) { return R > kTileRows * E; }

template <bool kPair, bool kGated>
cudaError_t launch(const GroupedArgs& g, const Args& a, cudaStream_t st) {
    using C = Cfg<kPair>;
    Maps maps;
    const uint64_t w_rows = static_cast<uint64_t>(g.E) * g.N;
    if (!encode_tmap_u8(&maps.x[0], g.xq, g.R, g.K, g.K, BK, kMinBox) ||
        !encode_tmap_u8(&maps.x[1], g.xq, g.R, g.K, g.K, BK, 2 * kMinBox) ||
        !encode_tmap_u8(&maps.x[2], g.xq, g.R, g.K, g.K, BK, 4 * kMinBox) ||
        !encode_tmap_u8(&maps.w, g.wq, w_rows, g.K, g.K, BK, kHalf) ||
        !encode_tmap_u8(&maps.w_small, g.wq, w_rows, g.K, g.K, BK, kHalf / 2))
        return cudaErrorInvalidValue;
    int ctas = g.num_sms < kMaxCtas ? g.num_sms : kMaxCtas;
    if (kPair && g.pair_clusters > 0 && 2 * g.pair_clusters < ctas) ctas = 2 * g.pair_clusters;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(ctas / C::CTAS * C::CTAS);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<kPair>();
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<kPair, kGated>, maps, a);
}

}  // namespace

size_t gemm_grouped_workspace(int64_t E, int64_t R, int64_t N, int64_t K) {
    (void)E, (void)N, (void)K;
    return static_cast<size_t>(kCountBytes + kMaxCtas * 2 * slot_floats(R) * 4);
}

int64_t gemm_grouped_zero_words() { return kCounts; }

cudaError_t prepare_gemm_grouped() {
    auto set = [](auto kernel, size_t bytes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    };
    cudaError_t e = set(gemm_grouped_kernel<false, false>, smem_bytes<false>());
    if (e == cudaSuccess) e = set(gemm_grouped_kernel<false, true>, smem_bytes<false>());
    if (e == cudaSuccess) e = set(gemm_grouped_kernel<true, false>, smem_bytes<true>());
    if (e == cudaSuccess) e = set(gemm_grouped_kernel<true, true>, smem_bytes<true>());
    return e;
}

cudaError_t launch_gemm_grouped(const GroupedArgs& g, cudaStream_t st) {
    Args a;
    a.s_tok = g.s_tok, a.s_w = g.s_w;
    a.offsets = g.offsets;
    a.y = static_cast<__nv_bfloat16*>(g.y);
    a.count = static_cast<unsigned*>(g.workspace);
    a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(g.workspace) + kCountBytes);
    a.slot = slot_floats(g.R);
    a.E = g.E, a.R = g.R, a.N = g.N, a.K = g.K;
    a.status = g.status;
    if (!g.zeroed) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, clear_counts, a.count, static_cast<int>(kCounts));
        if (e != cudaSuccess) return e;
    }
    // Measured: an SM alone streams 75 GB/s of weights (a stage is 32 KB), all together 6.1 TB/s;
    // a pair's stage takes the tensor cores 0.3 us; a part of 32 rows is added in 0.9 us, a pair's
    // in twice that, after 3 us for writing it and the counter.
    const int64_t mean = (static_cast<int64_t>(g.R) + g.E - 1) / g.E;
    const float batches = static_cast<float>((mean < kTileRows ? mean + 31 : kTileRows) / 32);
    a.costs.fixed = 3.0f;
    if (pairs_of(g.E, g.R)) {
        a.costs.stage = 0.3f, a.costs.shared = 0.0f, a.costs.part = 1.8f * batches;
        return g.swiglu ? launch<true, true>(g, a, st) : launch<true, false>(g, a, st);
    }
    a.costs.stage = 0.44f, a.costs.shared = 0.0054f, a.costs.part = 0.9f * batches;
    return g.swiglu ? launch<false, true>(g, a, st) : launch<false, false>(g, a, st);
}

}  // namespace fp8k
