// Causal attention over packed prompts, grouped heads, bf16:
//   out_i = sum_{j <= i} w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j - m_i)
// in one pass over the keys.  With the running maximum m and sum l of a row,
// a tile of keys adds
//   p_j = 2^(c s_j - c m),  l += sum_j p_j,  o += sum_j p_j v_j    (c = scale log2 e)
// and where a tile raises the maximum, l and o are first multiplied by
// 2^(c m_old - c m_new).  o only needs m to be near the maximum: it stays
// where it is until a tile exceeds it by 2^8 (p then reaches 256, which costs
// neither bf16 p nor the fp32 sums any digits), so o is rescaled a few times
// per row and not once per tile.
//
// Tiles.  A row is a (token, query head) pair: the G = Hq / Hkv query heads
// that share a key head lie next to one another, so a tile of 128 rows is
// 128 / G tokens with all their heads, keys and values are read once for the
// group, and short prompts fill the tile.  A CTA works on two such tiles (A
// and B) and walks over the keys in tiles of 128:
//   warps 0-3, 4-7  softmax of tile A and B: a thread holds a row of S (128
//                   fp32), writes P as bf16 over it, rescales O where needed
//                   and finally writes the row's output;
//   warp 8          TMA loads: Q once per item, K and V through a ring;
//   warp 9          issues the MMAs: S = Q K^T (both from shared memory) and
//                   O += P V (P from tensor memory);
//   warp 10         looks for infinities and NaN in values that some row of
//                   the item must not see (below).
// TMEM: S_A, S_B, O_A, O_B, 128 columns each: all 512.  While one tile is in
// its softmax the tensor core works on the other one.
//
// A masked weight is 0, but 0 * inf is NaN: in tiles where some row masks some
// key, warp 10 sets non-finite values to 0 in shared memory before the MMA
// reads them and remembers that it did; the rows that do see such a value get
// it back, from global memory, when they write their output.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace fp8k {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // log2 of how far p may exceed 1 before m moves
constexpr int kRows = 128;      // rows of a query tile
constexpr int kKeys = 128;      // keys of a tile
constexpr int kStages = 5;
constexpr int kThreads = 32 * 12;  // (warp 11 only fills up its warpgroup)
constexpr int kMainRegs = 208, kSideRegs = 88;  // 256 x 208 + 128 x 88 = 384 x 168, the launch's
constexpr int kClean = 4;       // (the ring holds two tiles of values at most)
constexpr int kFlags = 4;       // items whose "values were set to 0" flag is kept

struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t v_issued[kClean];  // such a tile of values is on its way (its stage's phase is current)
    uint64_t v_clean[kClean];   // warp 10 is done with it
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int dirty[kFlags];
};

template <int DP>
constexpr size_t smem_bytes() {
    return 1024 + (2 * kRows + kStages * kKeys) * DP * 2 + sizeof(Bars);
}

// A work item: the tokens of one sequence's block and one key head.
struct Item {
    int start, len;  // the sequence
    int q0;          // first token of the block, counted from the sequence's start
    int head;        // key head
    int tiles[2];    // key tiles of query tile A and B (0: empty)
    int masked;      // first key tile in which some row masks some key
    bool valid;
};

// Item `n` of the launch.  Blocks of `per` = 2 * tokens_per_tile tokens are
// numbered so that sequence b's begin at cu[b] / per + b (there is room for
// all of them, with some numbers unused), the last block first, since it has
// the most keys.
__device__ __forceinline__ Item find_item(int64_t n, int64_t blocks, const PromptArgs& a, int tpt) {
    Item it;
    const int64_t i = blocks - 1 - n / a.Hkv;
    it.head = static_cast<int>(n % a.Hkv);
    const int per = 2 * tpt;
    const int T = static_cast<int>(a.T);
    // the last sequence whose base is <= i: 32 candidates a step
    int64_t lo = 0, count = a.B;
    while (count > 1) {
        const int64_t step = (count + 31) / 32;
        const int64_t at = lo + step * lane_id();
        bool below = false;
        if (at < lo + count) {
            const int c = min(max(__ldg(a.cu + at), 0), T);
            below = c / per + at <= i;
        }
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, below);
        const int last = votes ? 31 - __clz(votes) : 0;
        const int64_t next = lo + step * last;
        count = min(step, lo + count - next);
        lo = next;
    }
    it.start = min(max(__ldg(a.cu + lo), 0), T);
    it.len = min(max(__ldg(a.cu + lo + 1), it.start), T) - it.start;
    const int64_t q0 = (i - (it.start / per + lo)) * per;
    it.valid = q0 >= 0 && q0 < it.len;
    it.q0 = static_cast<int>(q0);
    const int end_a = min(it.q0 + tpt, it.len), end_b = min(it.q0 + 2 * tpt, it.len);
    it.tiles[0] = (end_a + kKeys - 1) / kKeys;
    it.tiles[1] = it.q0 + tpt < it.len ? (end_b + kKeys - 1) / kKeys : 0;
    it.masked = it.q0 / kKeys;
    return it;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_prompt(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PromptArgs a, int64_t blocks) {
    constexpr int kCols = DP / 64;                 // 64-element columns of a tile
    constexpr uint32_t kColBytes = 128 * 128;      // 128 rows of 128 bytes
    constexpr uint32_t kTile = kCols * kColBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;                            // [2][kCols][128][128 B]
    uint8_t* sKV = smem + 2 * kTile;               // [kStages][kCols][128][128 B]
    Bars* bars = reinterpret_cast<Bars*>(sKV + kStages * kTile);
    const int warp = threadIdx.x >> 5, lane = lane_id();
    unsigned* status = a.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars->s_full[x], 1);
            mbar_init(&bars->p_full[x], 4);
            mbar_init(&bars->o_full[x], 1);
        }
        for (int k = 0; k < kClean; ++k) {
            mbar_init(&bars->v_issued[k], 1);
            mbar_init(&bars->v_clean[k], 1);
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        for (int f = 0; f < kFlags; ++f) bars->dirty[f] = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort;
    pdl_wait_primary();

    const int G = a.Hq / a.Hkv, tpt = kRows / G;
    const int64_t items = blocks * a.Hkv;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMainRegs));
        // ------------------------------------------------ softmax and output
        const int x = warp >> 2;                       // query tile A or B
        const int row = (warp & 3) * 32 + lane;
        const int tok = row / G, head_in = row - tok * G;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane quarter << 16
        const uint32_t tS = tmem + lanes + x * 128, tO = tmem + lanes + 256 + x * 128;
        const float c = a.scale * kLog2e;
        uint32_t s_phase = 0, o_phase = 0;
        int item_no = 0;
        bool ok = true;
        for (int64_t n = blockIdx.x; ok && n < items; n += gridDim.x) {
            const Item it = find_item(n, blocks, a, tpt);
            if (!it.valid) continue;
            const int my_tok = it.q0 + x * tpt + tok;
            const bool mine = tok < tpt && my_tok < it.len;
            const int tiles = it.tiles[x];
            float m = -INFINITY, l0 = 0.0f, l1 = 0.0f;
            for (int j = 0; j < tiles; ++j) {
                if (!(ok = warp_wait(&bars->s_full[x], s_phase, abort_flag, status))) break;
                s_phase ^= 1u;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld_32x32b_x32(tS + 32 * b, s[b]);
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld_wait_regs(s[b]);
                const int seen = my_tok - j * kKeys;   // keys 0 .. seen of the tile are seen
                if (seen < kKeys - 1) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * b + i > seen) s[b][i] = 0xFF800000u;  // -inf
                }
                float top[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    top[b] = __uint_as_float(s[b][0]);
#pragma unroll
                    for (int i = 1; i < 32; ++i) top[b] = fmaxf(top[b], __uint_as_float(s[b][i]));
                }
                const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // (m = -inf: the first keys that are seen set it)
                const bool raise = mine && (tile_top - m) * c > kSlack;
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    // (row by row, so that no row's digits depend on its neighbours)
                    const float next = raise ? tile_top : m;
                    const float keep = !raise ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - next) * c);
                    m = next;
                    l0 *= keep;
                    l1 *= keep;
                    if (j > 0) {
                        // S of tile j came after P V of tile j - 1: O is at rest
                        for (int b = 0; b < DP / 32; ++b) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(tO + 32 * b, o);
                            tmem_ld_wait_regs(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                            tmem_st_32x32b_x32(tO + 32 * b, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.0f : -m * c;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float y0 = base, y1 = base;
                        fma2(y0, y1, __uint_as_float(s[b][2 * i]), __uint_as_float(s[b][2 * i + 1]), c, c);
                        y0 = ex2(y0);
                        y1 = ex2(y1);
                        add2(l0, l1, y0, y1);
                        p[i] = pack_bf16(y0, y1);
                    }
                    tmem_st_32x32b_x16(tS + 16 * b, p);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[x]);
            }
            if (!ok) break;
            if (tiles > 0) {
                if (!(ok = warp_wait(&bars->o_full[x], o_phase, abort_flag, status))) break;
                o_phase ^= 1u;
                tc_fence_after();
                const float l = l0 + l1;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const int64_t t = it.start + my_tok;
                uint16_t* dst = a.out + t * a.ldo + static_cast<int64_t>(it.head * G + head_in) * a.D;
                const bool dirty = *reinterpret_cast<volatile int*>(&bars->dirty[item_no % kFlags]) != 0;
#pragma unroll 1
                for (int b = 0; b < DP / 32; ++b) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(tO + 32 * b, o);
                    tmem_ld_wait_regs(o);
                    if (!mine) continue;
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
                    if (dirty) {
                        for (int j = it.masked * kKeys; j <= my_tok; ++j) {
                            const uint16_t* v = a.v + (it.start + j) * a.ldv +
                                                static_cast<int64_t>(it.head) * a.D + 32 * b;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (32 * b + i < a.D) {
                                    const float e = __uint_as_float(static_cast<uint32_t>(v[i]) << 16);
                                    if (!isfinite(e)) f[i] += e;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (32 * b + 8 * i < a.D)
                            *reinterpret_cast<uint4*>(dst + 32 * b + 8 * i) = make_uint4(
                                pack_bf16(f[8 * i], f[8 * i + 1]), pack_bf16(f[8 * i + 2], f[8 * i + 3]),
                                pack_bf16(f[8 * i + 4], f[8 * i + 5]), pack_bf16(f[8 * i + 6], f[8 * i + 7]));
                    }
                }
            }
            ++item_no;
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSideRegs));
      if (warp == 8) {
        // ------------------------------------------------ TMA loads
        uint32_t stage = 0, phase = 0, q_phase = 0;
        uint32_t loads = 0, issued = 0;
        bool ok = true;
        auto tile = [&](const CUtensorMap* tm, int head, int tokens) {
            if (!(ok = warp_wait(&bars->empty[stage], phase ^ 1u, abort_flag, status))) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->full[stage], kTile);
                for (int x = 0; x < kCols; ++x)
                    tma_load_3d(sKV + stage * kTile + x * kColBytes, tm, &bars->full[stage], 64 * x,
                                head, tokens);
            }
            __syncwarp();
            ++loads;
            if (++stage == kStages) stage = 0, phase ^= 1u;
        };
        for (int64_t n = blockIdx.x; ok && n < items; n += gridDim.x) {
            const Item it = find_item(n, blocks, a, tpt);
            if (!it.valid) continue;
            if (!(ok = warp_wait(&bars->q_empty, q_phase ^ 1u, abort_flag, status))) break;
            q_phase ^= 1u;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->q_full, 2u * kCols * 128u * static_cast<uint32_t>(G * tpt));
                for (int x = 0; x < 2; ++x)
                    for (int y = 0; y < kCols; ++y)
                        tma_load_3d(sQ + x * kTile + y * kColBytes, &tmQ, &bars->q_full, 64 * y,
                                    it.head * G, it.start + it.q0 + x * tpt);
            }
            __syncwarp();
            const int tiles = max(it.tiles[0], it.tiles[1]);
            for (int j = 0; ok && j < tiles; ++j) {
                tile(&tmK, it.head, it.start + j * kKeys);
                if (ok) tile(&tmV, it.head, it.start + j * kKeys);
                if (ok && j >= it.masked) {
                    if (lane == 0) mbar_arrive(&bars->v_issued[issued % kClean]);
                    ++issued;
                }
            }
        }
        if (!ok) {  // gave up: let the copies in flight land before the memory goes
            const uint32_t back = loads < kStages ? loads : kStages;
            for (uint32_t i = 0; i < back; ++i) {
                const uint32_t k = loads - 1 - i;
                if (lane == 0) wait_landed(&bars->full[k % kStages], (k / kStages) & 1u, status);
            }
            if (lane == 0 && q_phase) wait_landed(&bars->q_full, q_phase ^ 1u, status);
            __syncwarp();
        }
      } else if (warp == 9) {
        // ------------------------------------------------ MMA
        constexpr uint32_t idS = idesc_f16(kRows, kKeys, true, false);
        constexpr uint32_t idO = idesc_f16(kRows, DP, true, true);
        uint32_t at = 0;  // stages consumed so far
        uint32_t q_phase = 0, p_phase[2] = {0, 0}, cleaned = 0;
        bool ok = true;
        auto landed = [&](uint32_t k) {
            ok = ok && warp_wait(&bars->full[k % kStages], (k / kStages) & 1u, abort_flag, status);
            return ok;
        };
        auto mma_s = [&](int x, uint32_t k) {
            if (lane == 0) {
                const uint64_t q = sdesc_kmajor_sw128(smem_u32(sQ + x * kTile));
                const uint64_t kd = sdesc_kmajor_sw128(smem_u32(sKV + (k % kStages) * kTile));
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    const uint32_t off = ((i / 4) * kColBytes + (i % 4) * 32) >> 4;
                    mma_f16(tmem + x * 128, q + off, kd + off, idS, i != 0);
                }
                mma_commit(&bars->s_full[x]);
            }
            __syncwarp();
        };
        auto mma_o = [&](int x, uint32_t k, bool first) {
            if (lane == 0) {
                const uint64_t vd = sdesc_nmajor_sw128(smem_u32(sKV + (k % kStages) * kTile), kColBytes);
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                    mma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + 8 * i, vd + i * (2048 >> 4), idO,
                               !(first && i == 0));
            }
            __syncwarp();
        };
        for (int64_t n = blockIdx.x; ok && n < items; n += gridDim.x) {
            const Item it = find_item(n, blocks, a, tpt);
            if (!it.valid) continue;
            const int tiles = max(it.tiles[0], it.tiles[1]);
            if (!(ok = warp_wait(&bars->q_full, q_phase, abort_flag, status))) break;
            q_phase ^= 1u;
            for (int j = 0; j <= tiles && ok; ++j) {
                const uint32_t kk = at + 2 * j, vv = at + 2 * j - 1;  // K of tile j, V of tile j - 1
                const bool more = j < tiles;
                if (more && !landed(kk)) break;
                if (j > 0) {
                    if (!landed(vv)) break;
                    if (j - 1 >= it.masked) {
                        if (!(ok = warp_wait(&bars->v_clean[cleaned % kClean], (cleaned / kClean) & 1u,
                                             abort_flag, status)))
                            break;
                        ++cleaned;
                    }
                }
                tc_fence_after();
                for (int x = 0; x < 2; ++x) {
                    if (j > 0 && j - 1 < it.tiles[x]) {
                        if (!(ok = warp_wait(&bars->p_full[x], p_phase[x], abort_flag, status))) break;
                        p_phase[x] ^= 1u;
                        tc_fence_after();
                        mma_o(x, vv, j == 1);
                        if (j == it.tiles[x] && lane == 0) mma_commit(&bars->o_full[x]);
                        __syncwarp();
                    }
                    if (j < it.tiles[x]) mma_s(x, kk);
                }
                if (!ok) break;
                if (lane == 0) {
                    if (j > 0) mma_commit(&bars->empty[vv % kStages]);
                    if (more) mma_commit(&bars->empty[kk % kStages]);
                    if (j + 1 == tiles) mma_commit(&bars->q_empty);
                }
                __syncwarp();
            }
            at += 2 * tiles;
        }
        if (lane == 0) {
            mma_commit(&bars->drain);
            wait_drain(&bars->drain, status);
        }
        __syncwarp();
      } else if (warp == 10) {
        // ------------------------------------------------ values that some row masks
        uint32_t at = 0, cleaned = 0;
        int item_no = 0;
        bool ok = true;
        for (int64_t n = blockIdx.x; ok && n < items; n += gridDim.x) {
            const Item it = find_item(n, blocks, a, tpt);
            if (!it.valid) continue;
            const int tiles = max(it.tiles[0], it.tiles[1]);
            bool dirty = false;
            for (int j = it.masked; j < tiles; ++j) {
                const uint32_t k = at + 2 * j + 1;
                if (!(ok = warp_wait(&bars->v_issued[cleaned % kClean], (cleaned / kClean) & 1u,
                                     abort_flag, status)) ||
                    !(ok = warp_wait(&bars->full[k % kStages], (k / kStages) & 1u, abort_flag, status)))
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
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP>
cudaError_t launch_dim(const PromptArgs& a, cudaStream_t st) {
    const int G = a.Hq / a.Hkv, tpt = kRows / G;
    const int64_t blocks = a.T / (2 * tpt) + a.B;
    CUtensorMap tq, tk, tv;
    const uint64_t T = static_cast<uint64_t>(a.T), D = static_cast<uint64_t>(a.D);
    if (!encode_tmap_heads(&tq, a.q, T, a.Hq, D, 2 * a.ldq, 64, G, tpt) ||
        !encode_tmap_heads(&tk, a.k, T, a.Hkv, D, 2 * a.ldk, 64, 1, kKeys) ||
        !encode_tmap_heads(&tv, a.v, T, a.Hkv, D, 2 * a.ldv, 64, 1, kKeys))
        return cudaErrorInvalidValue;
    const int64_t items = blocks * a.Hkv;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(items < a.num_sms ? items : a.num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<DP>();
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_prompt<DP>, tq, tk, tv, a, blocks);
}

}  // namespace

cudaError_t launch_attention_prompt(const PromptArgs& a, cudaStream_t st) {
    return a.D <= 64 ? launch_dim<64>(a, st) : launch_dim<128>(a, st);
}

cudaError_t prepare_attention_prompt() {
    const cudaError_t e = cudaFuncSetAttribute(attention_prompt<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes<64>()));
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(attention_prompt<128>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem_bytes<128>()));
}

}  // namespace fp8k
