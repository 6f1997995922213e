// Causal attention over packed prompts, grouped heads, bf16:
//   out_i = sum_{j <= i} w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j - m_i)
// in one pass over the keys (the softmax of a tile: attention_tile.cuh).
//
// Tiles.  A row is a (token, query head) pair: the G = Hq / Hkv query heads
// that share a key head lie next to one another, so a tile of 128 rows is
// 128 / G tokens with all their heads, keys and values are read once for the
// group, and short prompts fill the tile.  A CTA works on two such tiles (A
// and B; where prompts are short or few, on one, with two CTAs an SM) and
// walks over the keys in tiles of 128:
//   warps 0-7, 8-15 softmax of tile A and B: a warp holds 16 rows of S, four
//                   lanes a row, writes P as bf16 over S, rescales O where
//                   needed and finally writes the rows' output.  P has V's
//                   type, as an MMA's operands must: each weight is off by up
//                   to 2^-8 of itself, as the output is by its own rounding;
//                   their sum l is taken before that.  (Four warps a
//                   tile, a lane a row, took 1450 clocks a tile, mostly
//                   latency; the tensor core waits for S -> P of one tile
//                   once it is done with the other one's MMAs, 1024 clocks);
//   warp 16         finds the CTA's items and loads them by TMA: Q once per
//                   item, K and V through a ring.  The grid has a CTA for each
//                   item, the longest of a sequence first; a running CTA takes
//                   over the next one that has not started (cluster launch
//                   control), so that all end at about the same time;
//   warps 17, 19    issue the MMAs of tile A and of tile B: S = Q K^T (both
//                   from shared memory) and O += P V (P from tensor memory).
//                   They take turns, so that one tile is in its softmax while
//                   the tensor core has the other one (without turns the tiles
//                   fell into step and both waited).  An MMA takes the tensor
//                   core 64 clocks and a thread about 50 to issue, and a look
//                   at a barrier 100: a single issuer for both tiles took 2830
//                   clocks for 2048 clocks of MMAs.  P comes in two halves, the
//                   MMAs of the first 64 keys start with the first;
//   warp 18         looks for infinities and NaN in values that some row of
//                   the item must not see (below).
// (With one tile a CTA: softmax in warps 0-7, the others are warps 8-11.)
//
// Bound by the tensor cores where prompts are long.  Measured, heads of 128: one
// prompt of 8192 tokens, 32 / 8 heads, 335 to 345 us on a cool GPU, 365 to 380 back
// to back for seconds, 1.64 to 1.45 PFLOP/s, 86 to 76% of what a large library
// product reaches in a burst (tensor pipe 70% busy: the rest is the way S -> P ->
// O, 2600 to 3000 clocks for 2048 clocks of MMAs); nine prompts of 129 to 2801, 64 /
// 8 heads, 202 us, 1.18 PFLOP/s (an item's start and end take some 5000 clocks, in
// which the same warps write its output and take the next one's first softmax, and
// the masked halves of the last tiles are work too); 24 prompts of 1 to 257 tokens
// 17 us (items of two tiles: their latency).  Heads of 80, 96 and 112 run as heads
// of 128, on zeros: 4096 tokens 95, 96, 97 us, of 128 98, of 64 87.
//
// A masked weight is 0, but 0 * inf is NaN: in tiles where some row masks some
// key, warp 18 sets non-finite values to 0 in shared memory before the MMA
// reads them and remembers that it did; the rows that do see such a value get
// it back, from global memory, when they write their output.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "attention_tile.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr int kClean = 4;  // tiles of values with flags of their own
constexpr int kFlags = 4;  // items whose "values were set to 0" flag is kept

// A work item: the tokens of one sequence's block and one key head.
struct Item {
    int start, len;  // the sequence
    int q0;          // first token of the block, counted from the sequence's start
    int head;        // key head
    int tiles[2];    // key tiles of query tile A and B (0: empty)
    int masked;      // first key tile in which some row masks some key
    int valid;
};

// NQ: query tiles of a CTA.
template <int DP, int NQ>
struct Config {
    static constexpr int kStages = NQ == 2 ? 5 : 2;
    // (of stages in a row at most every other one and one more hold values)
    static_assert(kClean >= (kStages + 1) / 2, "a tile's flags must not meet the next one's");
    static constexpr int kMainWarps = 8 * NQ;
    static constexpr int kThreads = 32 * (kMainWarps + 4);
    static constexpr int kCtas = 3 - NQ;  // an SM
    // 512 x 104 + 128 x 64 = 640 x 96 and 256 x 96 + 128 x 48 = 384 x 80, the launch's
    static constexpr int kMainRegs = NQ == 2 ? 104 : 96, kSideRegs = NQ == 2 ? 64 : 48;
};

template <int kStages>
struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2], o_full[2];
    uint64_t v_issued[kClean];  // such a tile of values is on its way (its stage's phase is current)
    uint64_t v_clean[kClean];   // warp 18 is done with it
    uint64_t turn[2];  // an issuer may go on
    uint64_t drain[2];
    uint64_t item_full, item_empty, next_cta;
    alignas(16) uint4 response;  // of the request for the next item
    Item item;
    uint32_t tmem_base;
    int abort;
    int dirty[kFlags];
};

template <int DP, int NQ>
constexpr size_t smem_bytes() {
    using C = Config<DP, NQ>;
    return 1024 + (NQ * kRows + C::kStages * kKeys) * DP * 2 + sizeof(Bars<C::kStages>);
}

// Item `n` of the launch.  Blocks of `per` tokens are numbered so that
// sequence b's begin at cu[b] / per + b (there is room for all of them, with
// some numbers unused), the last block first, since it has the most keys.
__device__ __forceinline__ Item find_item(int64_t n, int64_t blocks, const PromptArgs& a, int tpt, int per) {
    Item it;
    const int64_t i = blocks - 1 - n / a.Hkv;
    it.head = static_cast<int>(n % a.Hkv);
    const int T = static_cast<int>(a.T);
    // the last sequence whose base is <= i: 32 candidates a step
    int64_t lo = 0, count = a.B;
    while (count > 1) {
        const int64_t step = (count + 31) / 32;
        const int64_t at = lo + step * lane_id();
        bool below = false;
        if (at < lo + count) {
            const int c = min(max(a.cu[at], 0), T);
            below = c / per + at <= i;
        }
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, below);
        const int last = votes ? 31 - __clz(votes) : 0;
        const int64_t next = lo + step * last;
        count = min(step, lo + count - next);
        lo = next;
    }
    it.start = min(max(a.cu[lo], 0), T);
    it.len = min(max(a.cu[lo + 1], it.start), T) - it.start;
    const int64_t q0 = (i - (it.start / per + lo)) * per;
    it.valid = q0 >= 0 && q0 < it.len;
    it.q0 = static_cast<int>(q0);
    const int end_a = min(it.q0 + tpt, it.len), end_b = min(it.q0 + per, it.len);
    it.tiles[0] = (end_a + kKeys - 1) / kKeys;
    it.tiles[1] = end_b > it.q0 + tpt ? (end_b + kKeys - 1) / kKeys : 0;
    it.masked = it.q0 / kKeys;
    return it;
}

// Adds to O the infinities and NaN of the values that a lane's rows see and
// that warp 18 took out of shared memory (rare, and slow): tokens `first` ..
// last of the sequence's values v.
template <int DP>
__device__ __noinline__ void add_unfinite(uint32_t tO, const uint16_t* v, int64_t ldv, int D, int first, int last0,
                                          int last1) {
    const int t = lane_id() & 3;
#pragma unroll 1
    for (int b = 0; b < DP / 32; ++b) {
        uint32_t o[16];
        __syncwarp();
        tmem_ld_16x256b_x4(tO + 32 * b, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(o[i]));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            for (int j = first; j <= (e ? last1 : last0); ++j) {
                const uint16_t* at = v + j * ldv + 32 * b + 2 * t;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = 8 * (i >> 1) + (i & 1);
                    if (32 * b + 2 * t + d < D) {
                        const float z = __uint_as_float(static_cast<uint32_t>(at[d]) << 16);
                        uint32_t& to = o[4 * (i >> 1) + 2 * e + (i & 1)];
                        if (!isfinite(z)) to = __float_as_uint(__uint_as_float(to) + z);
                    }
                }
            }
        }
        __syncwarp();
        tmem_st_16x256b_x4(tO + 32 * b, o);
    }
    tmem_st_wait();
}

// w[i] of lane t -> w[t] of lane i, within each quad of lanes.
__device__ __forceinline__ void transpose_quad(uint32_t (&w)[4], int t) {
    // the 2 x 2 blocks' off-diagonal, then within the blocks
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        const bool up = t & d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
            const uint32_t give = up ? w[i] : w[i | d];
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, d);
            if (up) w[i] = got; else w[i | d] = got;
        }
    }
}

template <int DP, int NQ>
__global__ void __launch_bounds__(Config<DP, NQ>::kThreads, Config<DP, NQ>::kCtas)
    attention_prompt(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PromptArgs a, int64_t blocks) {
    using C = Config<DP, NQ>;
    constexpr int kStages = C::kStages, kMainWarps = C::kMainWarps;
    constexpr uint32_t kTmem = 256 * NQ;           // columns: S of the tiles, then O
    constexpr int kCols = DP / 64;                 // 64-element columns of a tile
    constexpr uint32_t kColBytes = 128 * 128;      // 128 rows of 128 bytes
    constexpr uint32_t kTile = kCols * kColBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;                            // [NQ][kCols][128][128 B]
    uint8_t* sKV = smem + NQ * kTile;              // [kStages][kCols][128][128 B]
    auto* bars = reinterpret_cast<Bars<kStages>*>(sKV + kStages * kTile);
    const int warp = threadIdx.x >> 5, lane = lane_id();
    unsigned* status = a.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], NQ);  // (of each issuer)
        }
        for (int x = 0; x < NQ; ++x) {
            mbar_init(&bars->s_full[x], 1);
            mbar_init(&bars->p_full[x][0], 8);
            mbar_init(&bars->p_full[x][1], 8);
            mbar_init(&bars->o_full[x], 1);
            mbar_init(&bars->q_full[x], 1);
            mbar_init(&bars->q_empty[x], 1);
            mbar_init(&bars->turn[x], 1);
            mbar_init(&bars->drain[x], 1);
        }
        for (int k = 0; k < kClean; ++k) {
            mbar_init(&bars->v_issued[k], 1);
            mbar_init(&bars->v_clean[k], 1);
        }
        mbar_init(&bars->item_full, 1);
        mbar_init(&bars->item_empty, kMainWarps + 1 + NQ);
        mbar_init(&bars->next_cta, 1);
        bars->abort = 0;
        for (int f = 0; f < kFlags; ++f) bars->dirty[f] = 0;
        fence_mbar_init();
    }
    if (warp == kMainWarps && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == kMainWarps + 1) {
        tmem_alloc(&bars->tmem_base, kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();  // (behind the allocation: see ptx.cuh)
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort;
    pdl_wait_primary();

    const int G = a.Hq / a.Hkv, tpt = kRows / G;
    // The next item, for a whole warp: false where there is none (left).
    uint32_t items_taken = 0;
    auto take_item = [&](Item& it, bool& ok) {
        if (!(ok = warp_ready(&bars->item_full, items_taken & 1u, abort_flag, status))) return false;
        const volatile Item& from = bars->item;
        it.start = from.start, it.len = from.len, it.q0 = from.q0, it.head = from.head;
        it.tiles[0] = from.tiles[0], it.tiles[1] = from.tiles[1];
        it.masked = from.masked, it.valid = from.valid;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty);
        ++items_taken;
        return it.valid != 0;
    };

    if (warp < kMainWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMainRegs));
        // ------------------------------------------------ softmax and output
        const int x = warp >> 3, g = lane >> 2, t = lane & 3;  // query tile A or B
        const int row0 = (warp & 3) * 32 + (warp >> 2 & 1) * 16 + g;  // this lane's rows: row0, row0 + 8
        const uint32_t lanes = static_cast<uint32_t>(row0 - g) << 16;
        const uint32_t tS = tmem + lanes + x * 128, tO = tmem + lanes + kTmem / 2 + x * 128;
        const float c[2] = {a.scale * kLog2e, a.scale * kLog2e};
        uint32_t s_phase = 0, o_phase = 0;
        int item_no = 0;
        bool ok = true;
        int tok[2], head_in[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            tok[e] = (row0 + 8 * e) / G;
            head_in[e] = row0 + 8 * e - tok[e] * G;
        }
        Item it;
        while (ok && take_item(it, ok)) {
            int my_tok[2];
            bool mine[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                my_tok[e] = it.q0 + x * tpt + tok[e];
                mine[e] = tok[e] < tpt && my_tok[e] < it.len;
            }
            const int tiles = it.tiles[x];
            const int first_tok = it.q0 + x * tpt;  // no row of the tile sees less than this
            SoftmaxRows rows;
            for (int j = 0; j < tiles; ++j) {
                if (!(ok = warp_ready(&bars->s_full[x], s_phase, abort_flag, status))) break;
                s_phase ^= 1u;
                tc_fence_after();
                uint32_t s[4][16];
                load_scores(tS, s);
                if (first_tok - j * kKeys < kKeys - 1) {
                    hide_after(s, 0, my_tok[0] - j * kKeys - 2 * t);
                    hide_after(s, 1, my_tok[1] - j * kKeys - 2 * t);
                }
                softmax_tile<true, DP, true>(s, tS, tO, rows, c, mine, j > 0, [&](int h) {
                    if (lane == 0) mbar_arrive(&bars->p_full[x][h]);
                });
            }
            if (!ok) break;
            if (tiles > 0) {
                // (what needs no O comes before the wait for it)
                float inv[2];
                uint16_t* dst[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sum = rows.sum(e);
                    inv[e] = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
                    dst[e] = a.out + (it.start + my_tok[e]) * a.ldo +
                             static_cast<int64_t>(it.head * G + head_in[e]) * a.D + 8 * t;
                }
                if (!(ok = warp_ready(&bars->o_full[x], o_phase, abort_flag, status))) break;
                o_phase ^= 1u;
                tc_fence_after();
                if (*reinterpret_cast<volatile int*>(&bars->dirty[item_no % kFlags]) != 0)
                    add_unfinite<DP>(tO, a.v + it.start * a.ldv + static_cast<int64_t>(it.head) * a.D, a.ldv, a.D,
                                     it.masked * kKeys, mine[0] ? my_tok[0] : -1, mine[1] ? my_tok[1] : -1);
                uint32_t o[DP / 32][16];
#pragma unroll
                for (int b = 0; b < DP / 32; ++b) tmem_ld_16x256b_x4(tO + 32 * b, o[b]);
                tmem_ld_wait();
#pragma unroll
                for (int b = 0; b < DP / 32; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(o[b][i]));  // (no use before the wait)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int b = 0; b < DP / 32; ++b) {
                        // w[i]: elements 8 i + 2 t, + 1; the quad's lanes exchange them so
                        // that lane t has elements 8 t .. 8 t + 7 for one 16-byte store
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float y0, y1;
                            mul2(y0, y1, __uint_as_float(o[b][4 * i + 2 * e]),
                                 __uint_as_float(o[b][4 * i + 2 * e + 1]), inv[e], inv[e]);
                            w[i] = pack_bf16(y0, y1);
                        }
                        transpose_quad(w, t);
                        if (mine[e] && 32 * b + 8 * t < a.D)
                            *reinterpret_cast<uint4*>(dst[e] + 32 * b) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
            }
            ++item_no;
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kSideRegs));
      if (warp == kMainWarps) {
        // ------------------------------------------------ TMA loads
        uint32_t loads = 0, issued = 0, q_loads = 0, q_issued[2] = {0, 0}, published = 0, asked = 0, answered = 0;
        bool ok = true;
        Item it;
        auto ask = [&]() {
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->next_cta, 16);
                cancel_next_cta(&bars->response, &bars->next_cta);
            }
            ++asked;
            __syncwarp();
        };
        auto answer = [&](int64_t& n) {
            if (!warp_ready(&bars->next_cta, answered & 1u, abort_flag, status)) return false;
            ++answered;
            n = cancelled_cta(&bars->response);
            fence_proxy_async_smem();  // (read, before the next answer is written)
            __syncwarp();
            return true;
        };
        auto publish = [&]() {  // (an invalid item tells that there are no more)
            if (!warp_ready(&bars->item_empty, (published & 1u) ^ 1u, abort_flag, status)) return false;
            if (lane == 0) bars->item = it;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->item_full);
            ++published;
            return true;
        };
        auto tile = [&](const CUtensorMap* tm, int head, int tokens) {
            const uint32_t stage = loads % kStages;
            if (!wait_bounded(&bars->empty[stage], (loads / kStages & 1u) ^ 1u, abort_flag, status))
                return false;
            mbar_arrive_expect_tx(&bars->full[stage], kTile);
            for (int y = 0; y < kCols; ++y)
                tma_load_3d(sKV + stage * kTile + y * kColBytes, tm, &bars->full[stage], 64 * y, head,
                            tokens);
            ++loads;
            return true;
        };
        auto queries = [&](int x) {
            if (!wait_bounded(&bars->q_empty[x], (q_loads & 1u) ^ 1u, abort_flag, status)) return false;
            mbar_arrive_expect_tx(&bars->q_full[x], kCols * 128u * static_cast<uint32_t>(G * tpt));
            for (int y = 0; y < kCols; ++y)
                tma_load_3d(sQ + x * kTile + y * kColBytes, &tmQ, &bars->q_full[x], 64 * y, it.head * G,
                            it.start + it.q0 + x * tpt);
            ++q_issued[x];
            return true;
        };
        auto load_item = [&]() {
            const int tiles = max(it.tiles[0], it.tiles[1]);
            for (int j = 0; j < tiles; ++j) {
                // the queries of tile A are wanted first: before the last turn's of tile B are done with
                if (j == 0 && !queries(0)) return false;
                if (!tile(&tmK, it.head, it.start + j * kKeys)) return false;
                if (j == 0 && NQ == 2 && !queries(1)) return false;
                if (j == 0) ++q_loads;
                if (!tile(&tmV, it.head, it.start + j * kKeys)) return false;
                if (j >= it.masked) {
                    mbar_arrive(&bars->v_issued[issued % kClean]);
                    ++issued;
                }
            }
            return true;
        };
        int64_t n = blockIdx.x;
        while (true) {
            // the next item: its number may belong to no block of any sequence
            while (n >= 0 && !(it = find_item(n, blocks, a, tpt, NQ * tpt)).valid) {
                ask();
                if (!(ok = answer(n))) break;
            }
            if (!ok) break;
            if (n < 0) it.valid = 0;
            if (!(ok = publish()) || n < 0) break;
            ask();  // (answered while this one is loaded)
            if (lane == 0) ok = load_item();
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            if (!(ok = answer(n))) break;
        }
        if (!ok && lane == 0) {  // gave up: let the copies in flight land before the memory goes
            for (uint32_t i = 1; i <= kStages && i <= loads; ++i) {
                const uint32_t k = loads - i;
                wait_landed(&bars->full[k % kStages], k / kStages & 1u, status);
            }
            for (int x = 0; x < NQ; ++x)
                if (q_issued[x]) wait_landed(&bars->q_full[x], (q_issued[x] - 1) & 1u, status);
            if (asked != answered) wait_landed(&bars->next_cta, answered & 1u, status);
        }
        __syncwarp();
      } else if (warp == kMainWarps + 1 || (NQ == 2 && warp == kMainWarps + 3)) {
        // ------------------------------------------------ MMA
        const int x = uniform(warp == kMainWarps + 1 ? 0 : 1);  // query tile A or B
        constexpr uint32_t idS = idesc_f16(kRows, kKeys, true, false);
        constexpr uint32_t idO = idesc_f16(kRows, DP, true, true);
        // (the warp stays converged and every operand of an MMA is uniform: see elect_one)
        const uint32_t tm = uniform(tmem);
        const uint32_t base_q = uniform(smem_u32(sQ)), base_kv = uniform(smem_u32(sKV));
        uint32_t at = 0;  // stages consumed so far
        uint32_t q_phase = 0, p_phase = 0, cleaned = 0, turns = 0;
        bool ok = true;
        const uint32_t tS = tm + x * 128, tO = tm + kTmem / 2 + x * 128;
        const uint32_t qd = desc_kmajor(base_q + x * kTile);
        auto ready = [&](uint64_t* bar, uint32_t parity) {
            return warp_ready(bar, parity & 1u, abort_flag, status);
        };
        auto landed = [&](uint32_t k) { return ready(&bars->full[k % kStages], k / kStages); };
        Item it;
        while (ok && take_item(it, ok)) {
            const int tiles = uniform(max(it.tiles[0], it.tiles[1])), masked = uniform(it.masked);
            const int mine = uniform(it.tiles[x]);
            if (!(ok = ready(&bars->q_full[x], q_phase))) break;
            q_phase ^= 1u;
            for (int j = 0; j <= tiles; ++j) {
                // P V of key tile j - 1 and S of key tile j.  All looks at barriers but one
                // come before the turn, all looks ahead after it.
                const uint32_t kk = (at + 2 * j) % kStages, vv = (at + 2 * j + kStages - 1) % kStages;
                const uint32_t kd = desc_kmajor(base_kv + uniform(kk) * kTile);
                const uint32_t vd = desc_nmajor(base_kv + uniform(vv) * kTile, kColBytes);
                const bool pv = j > 0 && j - 1 < mine;
                if (j < tiles && !(ok = landed(at + 2 * j))) break;
                if (pv && !(ok = ready(&bars->p_full[x][0], p_phase))) break;
                if (NQ == 2) {
                    if (!(ok = ready(&bars->turn[x], x == 0 ? turns ^ 1u : turns))) break;
                    turns ^= 1u;
                }
                tc_fence_after();
                if (pv) {
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_f16_ts(tO, tS + 8 * i, vd + i * (2048 >> 4), idO, !(j == 1 && i == 0));
                    }
                    __syncwarp();
                    if (!(ok = ready(&bars->p_full[x][1], p_phase))) break;
                    p_phase ^= 1u;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 4; i < 8; ++i) mma_f16_ts(tO, tS + 8 * i, vd + i * (2048 >> 4), idO, 1);
                        if (j == mine) mma_commit(&bars->o_full[x]);
                    }
                    __syncwarp();
                }
                if (j < mine) {
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) {
                            const uint32_t off = ((i / 4) * kColBytes + (i % 4) * 32) >> 4;
                            mma_f16(tS, qd + off, kd + off, idS, i != 0);
                        }
                        mma_commit(&bars->s_full[x]);
                    }
                    __syncwarp();
                }
                if (elect_one()) {
                    if (NQ == 2) mbar_arrive(&bars->turn[x ^ 1]);
                    if (j > 0) mma_commit(&bars->empty[vv]);
                    if (j < tiles) mma_commit(&bars->empty[kk]);
                    if (j + 1 == tiles) mma_commit(&bars->q_empty[x]);
                }
                __syncwarp();
                if (j < tiles) {
                    if (!(ok = landed(at + 2 * j + 1))) break;
                    if (j >= masked) {
                        if (!(ok = ready(&bars->v_clean[cleaned % kClean], cleaned / kClean))) break;
                        ++cleaned;
                    }
                }
            }
            if (!ok) break;
            at += 2 * tiles;
        }
        __syncwarp();
        if (elect_one()) {  // (the lane that issued the MMAs)
            mma_commit(&bars->drain[x]);
            wait_drain(&bars->drain[x], status);
        }
        __syncwarp();
      } else if (warp == kMainWarps + 2) {
        // ------------------------------------------------ values that some row masks
        uint32_t at = 0, cleaned = 0;
        int item_no = 0;
        bool ok = true;
        Item it;
        while (ok && take_item(it, ok)) {
            const int tiles = max(it.tiles[0], it.tiles[1]);
            bool dirty = false;
            for (int j = it.masked; j < tiles; ++j) {
                const uint32_t k = at + 2 * j + 1;
                if (!(ok = warp_ready(&bars->v_issued[cleaned % kClean], (cleaned / kClean) & 1u,
                                     abort_flag, status)) ||
                    !(ok = warp_ready(&bars->full[k % kStages], (k / kStages) & 1u, abort_flag, status)))
                    break;
                uint4* v = reinterpret_cast<uint4*>(sKV + (k % kStages) * kTile);
                uint32_t found = 0;
#pragma unroll 8
                for (int i = lane; i < static_cast<int>(kTile / 16); i += 32) {
                    const uint4 u = v[i];
                    // an exponent of all ones carries into the halfword's top bit
                    found |= ((u.x & 0x7F807F80u) + 0x00800080u) | ((u.y & 0x7F807F80u) + 0x00800080u) |
                             ((u.z & 0x7F807F80u) + 0x00800080u) | ((u.w & 0x7F807F80u) + 0x00800080u);
                }
                if (__any_sync(0xFFFFFFFFu, (found & 0x80008000u) != 0)) {
                    dirty = true;
                    uint16_t* e = reinterpret_cast<uint16_t*>(v);
                    for (int i = lane; i < static_cast<int>(kTile / 2); i += 32)
                        if ((e[i] & 0x7F80u) == 0x7F80u) e[i] = 0;
                    fence_proxy_async_smem();
                }
                if (lane == 0) {
                    // (the flag before the last arrival: O is complete after it)
                    *reinterpret_cast<volatile int*>(&bars->dirty[item_no % kFlags]) = dirty ? 1 : 0;
                    __threadfence_block();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->v_clean[cleaned % kClean]);
                ++cleaned;
            }
            at += 2 * tiles;
            ++item_no;
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMainWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

template <int DP, int NQ>
cudaError_t launch_tiles(const PromptArgs& a, cudaStream_t st) {
    using C = Config<DP, NQ>;
    const int G = a.Hq / a.Hkv, tpt = kRows / G;
    const int64_t blocks = a.T / (NQ * tpt) + a.B, items = blocks * a.Hkv;
    if (items > INT32_MAX) return cudaErrorInvalidConfiguration;
    CUtensorMap tq, tk, tv;
    const uint64_t T = static_cast<uint64_t>(a.T), D = static_cast<uint64_t>(a.D);
    if (!encode_tmap_heads(&tq, a.q, T, a.Hq, D, 2 * a.ldq, 64, G, tpt) ||
        !encode_tmap_heads(&tk, a.k, T, a.Hkv, D, 2 * a.ldk, 64, 1, kKeys) ||
        !encode_tmap_heads(&tv, a.v, T, a.Hkv, D, 2 * a.ldv, 64, 1, kKeys))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(items));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem_bytes<DP, NQ>();
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_prompt<DP, NQ>, tq, tk, tv, a, blocks);
}

template <int DP, int NQ>
cudaError_t prepare() {
    return cudaFuncSetAttribute(attention_prompt<DP, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem_bytes<DP, NQ>()));
}

}  // namespace

cudaError_t launch_attention_prompt(const PromptArgs& a, cudaStream_t st) {
    // Too few items for the SMs: smaller ones.  (32 heads on 8 of 128: one prompt
    // of 128 tokens 6.9 us with one tile a CTA, 9.0 with two; of 1024 tokens 23.2
    // and 18.7, of 4096 tokens 126 and 98.)  Prompts that as a rule leave the
    // second tile empty: the same (128 of 32 tokens 28.8 and 34.6, 256 of 16 42 and
    // 54, 64 of 64 27.1 and 27.4, 16 of 257 34.7 and 33.6).
    const int64_t per = 2 * (kRows / (a.Hq / a.Hkv));  // tokens of two tiles
    const bool one = (a.T / per + a.B) * a.Hkv <= a.num_sms / 2 || a.T <= a.B * per;
    if (a.D <= 64) return one ? launch_tiles<64, 1>(a, st) : launch_tiles<64, 2>(a, st);
    return one ? launch_tiles<128, 1>(a, st) : launch_tiles<128, 2>(a, st);
}

cudaError_t prepare_attention_prompt() {
    for (cudaError_t e : {prepare<64, 1>(), prepare<64, 2>(), prepare<128, 1>(), prepare<128, 2>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace fp8k
