// The shared-prefix part of decode attention: the queries of all requests
// against tokens that all of them share, which are read once for all.
//
//   s = q . k,  p = 2^(c s - c m + 7),  o = sum p v   (attention_tile.cuh; c = scale
//                                                      log2(e) k_scale of the row)
//
// With B requests this is a product of B G query rows a key head with the
// prefix, bound by the tensor cores once B G is some 100 rows, where reading
// the prefix anew for each request would be bound by B times its bytes.  So
// it runs like prompt attention: tiles of 128 rows (128 / G requests with all
// heads of the group), two of them a CTA, key tiles of 128, S, P and O in
// tensor memory.  What differs:
//   * keys and values are E4M3 in pages.  Seven warps (17-23) bring them in 32
//     tokens at a time: a page look-up a token, asynchronous copies of the
//     codes into a buffer of the warp's own, conversion to f16, which is
//     exact, and a store to shared memory in the layout that the MMA reads.
//     (Three warps that kept the codes in registers took 7 us a tile);
//   * queries go to f16 with their exponent taken out (query_shift), P is f16;
//   * the prefix is cut into parts so that the CTAs fill the SMs; the CTAs of a
//     cluster have parts of the same rows, and add them up through
//     distributed shared memory: one (m, l, o) a row and cluster goes to the
//     workspace, from where the decode kernel goes on.  (With a part a CTA the
//     decode kernel spent 7 us a request on 16 of them.)
//
// Measured: 64 requests, 32 / 8 heads of 128, 8192 tokens shared and 1 to 777 of
// their own: 39 us with the kernels after it; 121 without this one.  Its 20 us
// are 2.3 until the first codes are asked for, 3 until S of the first key tile
// is there, 2 a key tile (two softmaxes in turn, each slowed to 2600 clocks by the
// load warps beside them, which take 3000 for 32 tokens and wait for nothing), 1
// for the last P V, 2.5 to have all parts of a cluster in shared
// memory and 4.3 to add them up (128 KB a CTA, three quarters from other SMs; the
// order and the number of loads on their way make no difference).
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_plan.h"
#include "attention_tile.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

constexpr int kStages = kPrefixStages;
constexpr int kMainWarps = 16;                 // softmax: 8 a query tile
constexpr int kLoadWarps = 7;
constexpr int kMainRegs = 88, kSideRegs = 64;  // 512 x 88 + 256 x 64 = 768 x 80, the launch's
constexpr int kThreads = 32 * (kMainWarps + 1 + kLoadWarps);

struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full;
    uint64_t s_full[2], p_full[2][2], o_full[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    uint32_t there[kThereRows][4];  // which tokens of a key tile exist: there_row()
    int lost_from;               // first key tile of this CTA whose values lost NaN
    float2 ml[2 * kRows];        // (m, l) of this CTA's part, m in log2 units
};

template <int DP>
constexpr size_t smem_bytes() {
    return 1024 + (2 * kRows + kStages * kKeys) * DP * 2 + kLoadWarps * 32 * DP + sizeof(Bars);
}

// Byte offset of 16-byte chunk `c` (of DP / 8) of row r in a tile of 128 rows:
// columns of 64 elements, 128-byte rows, chunks permuted by the row.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// NaN codes among the 16 E4M3 values at `addr` in shared memory become zeros;
// whether there were any.
__device__ __forceinline__ bool take_nan(uint32_t addr) {
    const uint4 u = ld_shared16(addr);
    uint32_t w[4] = {u.x, u.y, u.z, u.w}, found = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (seven ones carry into the byte's top bit)
        const uint32_t nan = ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
        found |= nan;
        w[i] &= ~((nan >> 7) * 0xFFu);
    }
    if (found) st_shared16(addr, w[0], w[1], w[2], w[3]);
    return found != 0;
}

// Gives O back the NaN of the values that a lane's rows see and that the load
// warps took out (rare, and slow): of tokens `from` .. to - 1, values v.  (Out of
// line: in the kernel's own code it cost 0.5 to 3 us of 39 without ever running.)
template <int DP>
__device__ __noinline__ void add_nan(uint32_t tO, const uint8_t* v, int64_t row_bytes, int D, const int32_t* table,
                                     unsigned page, int64_t n_pages, int from, int to0, int to1) {
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
            for (int tok = from; tok < (e ? to1 : to0); ++tok) {
                const unsigned pg = static_cast<unsigned>(tok) / page;
                const int id = table[pg];
                if (id < 0 || id >= n_pages) continue;
                const uint8_t* at = v + (id * static_cast<int64_t>(page) + (tok - pg * page)) * row_bytes + 32 * b + 2 * t;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = 8 * (i >> 1) + (i & 1);
                    if (32 * b + 2 * t + d < D && (at[d] & 0x7Fu) == 0x7Fu)
                        o[4 * (i >> 1) + 2 * e + (i & 1)] = 0x7FFFFFFFu;
                }
            }
        }
        __syncwarp();
        tmem_st_16x256b_x4(tO + 32 * b, o);
    }
    tmem_st_wait();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) attention_prefix(const DecodeArgs a, const PrefixPlan plan) {
    constexpr uint32_t kColBytes = 128 * 128;
    constexpr uint32_t kTile = DP / 64 * kColBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sQ = smem_u32(smem), sKV = sQ + 2 * kTile;
    const uint32_t sRaw = sKV + kStages * kTile;  // the load warps' codes
    Bars* bars = reinterpret_cast<Bars*>(smem + (2 + kStages) * kTile + kLoadWarps * 32 * DP);
    const int warp = threadIdx.x >> 5, lane = lane_id();
    unsigned* status = a.status;

    if (threadIdx.x < 2 * kRows) bars->ml[threadIdx.x] = make_float2(-INFINITY, 0.0f);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->full[s], 4);  // 32 tokens each
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->q_full, kMainWarps);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars->s_full[x], 1);
            mbar_init(&bars->p_full[x][0], kMainWarps / 2);
            mbar_init(&bars->p_full[x][1], kMainWarps / 2);
            mbar_init(&bars->o_full[x], 1);
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        bars->lost_from = INT32_MAX;
        fence_mbar_init();
    }
    if (warp == kMainWarps) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();  // (behind the allocation: see ptx.cuh)
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort;
    pdl_wait_primary();

    // this CTA's part of the prefix, key head and requests
    const int split = static_cast<int>(blockIdx.x % plan.splits);
    const int64_t rest = blockIdx.x / plan.splits;
    const int hk = static_cast<int>(rest % a.Hkv);
    const int64_t block = rest / a.Hkv;
    const int G = a.Hq / a.Hkv, tpt = kRows / G;
    const int64_t b0 = block * 2 * tpt;  // first request of tile A; B: b0 + tpt
    const int tile0 = split * plan.tiles;
    const int all_tiles = static_cast<int>((a.prefix + kKeys - 1) / kKeys);
    const int tiles = max(min(plan.tiles, all_tiles - tile0), 0);
    const bool two = b0 + tpt < a.B;     // tile B has requests

    if (warp < kMainWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMainRegs));
        // ------------------------------------------------ queries, softmax, output
        const int x = warp >> 3, g = lane >> 2, t = lane & 3;
        const int row0 = (warp & 3) * 32 + (warp >> 2 & 1) * 16 + g;
        const uint32_t lanes = static_cast<uint32_t>(row0 - g) << 16;
        const uint32_t tS = tmem + lanes + x * 128, tO = tmem + lanes + 256 + x * 128;
        const float unit = a.scale * kLog2e * a.k_scale[hk * a.scale_stride];
        float c[2];
        bool real[2];
        int limit[2], least = static_cast<int>(a.prefix);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row0 + 8 * e, tok = r / G;
            const int64_t b = b0 + x * tpt + tok;
            real[e] = tok < tpt && b < a.B;
            limit[e] = real[e] ? max(0, min(a.lens[b], static_cast<int>(a.prefix))) : static_cast<int>(a.prefix);
            least = min(least, limit[e]);
            uint4 u[DP / 32];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int ch = 4 * i + t;
                u[i] = make_uint4(0, 0, 0, 0);
                if (real[e] && 8 * ch < a.D)
                    u[i] = *reinterpret_cast<const uint4*>(
                        a.q + b * a.ldq + static_cast<int64_t>(hk * G + (r - tok * G)) * a.D + 8 * ch);
                top = top_of(u[i], top);
            }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int shift = query_shift(top);
            // (never 0, which would make -inf of a masked score and the first maximum NaN;
            // |s| < 2^31, so below 2^-126 all weights of the row are 1 anyhow)
            c[e] = scaled(unit, -shift);
            if (fabsf(c[e]) < 0x1p-126f) c[e] = 0x1p-126f;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = pack_f16(scaled(bf16lo(w[k]), shift), scaled(bf16hi(w[k]), shift));
                st_shared16(sQ + x * kTile + tile_chunk(r, 4 * i + t), h[0], h[1], h[2], h[3]);
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, d));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);

        SoftmaxRows rows;
        bool ok = true;
        if (tiles > 0 && (x == 0 || two)) {
            for (int j = 0; j < tiles; ++j) {
                if (!(ok = warp_ready(&bars->s_full[x], j & 1, abort_flag, status))) break;
                tc_fence_after();
                uint32_t s[4][16];
                load_scores(tS, s);
                const int key0 = (tile0 + j) * kKeys + 2 * t;
                if ((tile0 + j + 1) * kKeys > least) {
                    hide_after(s, 0, limit[0] - 1 - key0);
                    hide_after(s, 1, limit[1] - 1 - key0);
                }
                const volatile uint32_t* there = bars->there[there_row(j)];
                const uint32_t word[4] = {there[0], there[1], there[2], there[3]};
                if ((word[0] & word[1] & word[2] & word[3]) != 0xFFFFFFFFu) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (!(word[b] >> (2 * t + 8 * (i >> 1) + (i & 1)) & 1u))
                                s[b][4 * (i >> 1) + (i & 1)] = s[b][4 * (i >> 1) + 2 + (i & 1)] = 0xFF800000u;
                }
                softmax_tile<false, DP, false>(s, tS, tO, rows, c, real, j > 0, [&](int h) {
                    if (lane == 0) mbar_arrive(&bars->p_full[x][h]);
                });
            }
            if (ok && (ok = warp_ready(&bars->o_full[x], 0, abort_flag, status))) {
                tc_fence_after();
                const int lost = *reinterpret_cast<volatile int*>(&bars->lost_from);
                if (lost < tiles) {
                    const int end = (tile0 + tiles) * kKeys;
                    add_nan<DP>(tO, a.v_cache + static_cast<int64_t>(hk) * a.D, static_cast<int64_t>(a.Hkv) * a.D, a.D,
                                a.table, static_cast<unsigned>(a.page), a.n_pages, (tile0 + lost) * kKeys,
                                real[0] ? min(limit[0], end) : 0, real[1] ? min(limit[1], end) : 0);
                }
                // Tile A's part goes where the queries were (S of both tiles is complete by
                // now), B's where keys and values were (it is the last MMA that reads them).
                float* part = reinterpret_cast<float*>(smem + (x == 0 ? 0 : 2 * kTile));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sum = rows.sum(e);
                    if (t == 0)
                        bars->ml[x * kRows + row0 + 8 * e] =
                            make_float2(rows.m[e] == -INFINITY ? -INFINITY : rows.m[e] * c[e], sum);
                }
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
                        // (16-byte chunks permuted by the row, against bank conflicts)
                        float* dst = part + (row0 + 8 * e) * DP;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ch = (8 * b + 2 * i + (t >> 1)) ^ (row0 & 7);
                            *reinterpret_cast<float2*>(dst + 4 * ch + 2 * (t & 1)) = make_float2(
                                __uint_as_float(o[4 * i + 2 * e]), __uint_as_float(o[4 * i + 2 * e + 1]));
                        }
                    }
                }
                __syncwarp();
            }
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSideRegs));
      if (warp == kMainWarps) {
        // ------------------------------------------------ MMA
        constexpr uint32_t idS = idesc_f16(kRows, kKeys, false, false);
        constexpr uint32_t idO = idesc_f16(kRows, DP, false, true);
        // (the warp stays converged and every operand of an MMA is uniform: see elect_one)
        const uint32_t tm = uniform(tmem), base_q = uniform(sQ), base_kv = uniform(sKV);
        const int n = uniform(tiles), both = uniform(two ? 2 : 1);
        auto ready = [&](uint64_t* bar, uint32_t parity) {
            return warp_ready(bar, parity & 1u, abort_flag, status);
        };
        auto landed = [&](uint32_t k) { return ready(&bars->full[k % kStages], k / kStages); };
        bool ok = n > 0 && ready(&bars->q_full, 0) && landed(0);
        for (int j = 0; ok && j <= n; ++j) {
            // P V of tile j - 1 and S of tile j; what they read is there
            const uint32_t kk = key_stage(j), vv = value_stage(j - 1);  // (j = 0: not used)
            const uint32_t kd = desc_kmajor(base_kv + uniform(kk) * kTile);
            const uint32_t vd = desc_nmajor(base_kv + uniform(vv) * kTile, kColBytes);
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x < both) {
                    const uint32_t dS = tm + x * 128, dO = tm + 256 + x * 128;
                    const uint32_t qd = desc_kmajor(base_q + x * kTile);
                    if (j > 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(ok = ready(&bars->p_full[x][h], j - 1))) break;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int i = 4 * h; i < 4 * h + 4; ++i)
                                    mma_f16_ts(dO, dS + 8 * i, vd + i * (2048 >> 4), idO, !(j == 1 && i == 0));
                                if (h == 1 && j == n) mma_commit(&bars->o_full[x]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                    if (j < n) {
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < DP / 16; ++i) {
                                const uint32_t off = ((i / 4) * kColBytes + (i % 4) * 32) >> 4;
                                mma_f16(dS, qd + off, kd + off, idS, i != 0);
                            }
                            mma_commit(&bars->s_full[x]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok) break;
            if (elect_one()) {
                if (j > 0) mma_commit(&bars->empty[vv]);
                if (j < n) mma_commit(&bars->empty[kk]);
            }
            __syncwarp();
            if (j + 1 < n && !(ok = landed(2 * j + 2))) break;
            if (j < n && !(ok = landed(2 * j + 1))) break;
        }
        __syncwarp();
        if (elect_one()) {
            mma_commit(&bars->drain);
            wait_drain(&bars->drain, status);
        }
        __syncwarp();
      } else {
        // ------------------------------------------------ codes -> f16 tiles
        constexpr int kChunks = DP / 16;  // 16-code chunks of a token
        const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * a.D;
        const unsigned page = static_cast<unsigned>(a.page);
        const int jobs = 8 * tiles;  // job 8 j + q: keys of tokens 32 q + ... of key tile j; + 4: their values
        // the slot of this lane's token of a job; -1: none, or not in the prefix
        auto slot_of = [&](int job) {
            const int64_t tok = static_cast<int64_t>(tile0 + (job >> 3)) * kKeys + 32 * (job & 3) + lane;
            if (job >= jobs || tok >= a.prefix) return -1;
            const unsigned pg = static_cast<unsigned>(tok) / page;
            const int id = a.table[pg];
            if (id < 0 || id >= a.n_pages) return -1;
            return static_cast<int>(id * page + (static_cast<unsigned>(tok) - pg * page));
        };
        const uint32_t raw = sRaw + (warp - kMainWarps - 1) * 32 * DP;
        const uint32_t ch = lane % kChunks;
        // Half a job's codes at a time, so that one half is on its way while the
        // other one is converted.
        auto copy = [&](int job, int slots, int h) {
            const uint8_t* from = (job & 4 ? a.v_cache : a.k_cache) + static_cast<int64_t>(hk) * a.D + 16 * ch;
#pragma unroll
            for (int i = h * kChunks / 2; i < (h + 1) * kChunks / 2; ++i) {
                const int s = __shfl_sync(0xFFFFFFFFu, slots, (32 * i + lane) / kChunks);
                copy_async16(raw + 512 * i + 16 * lane, from + s * row_bytes, s >= 0 && 16 * ch < a.D);
            }
            copy_commit();
        };
        // where this lane's chunks go in a tile: the first of the job's row
        // lane / kChunks and of the next row that another permutation meets
        constexpr int kStep = 32 / kChunks;           // rows between two chunks of a lane
        const int r0 = lane / kChunks;
        // (of eight lanes with one row, four store their second half first: with the
        // first halves alone each bank would be met twice; 256 requests, 16384 tokens,
        // 64 / 8 heads: 197 us instead of 202)
        const bool swap = kChunks == 8 && ch >= 4;
        const uint32_t c0 = 2 * ch + (swap ? 1 : 0), c1 = 2 * ch + (swap ? 0 : 1);
        const uint32_t at[2][2] = {{tile_chunk(r0, c0), tile_chunk(r0, c1)},
                                   {tile_chunk(r0 + kStep, c0), tile_chunk(r0 + kStep, c1)}};
        int job = warp - kMainWarps - 1;
        int now = slot_of(job), next = slot_of(job + kLoadWarps);
        if (job < jobs) {
            copy(job, now, 0);
            copy(job, now, 1);
        }
        // The tokens that every request of this CTA sees.  Beyond them a weight may be
        // 0 beside a value that is NaN, and 0 NaN is NaN: there such values are set to 0,
        // and the rows that see them get them back with their output.
        int all_see = static_cast<int>(a.prefix);
        for (int64_t b = b0 + lane; b < min(b0 + 2 * tpt, a.B); b += 32) all_see = min(all_see, max(a.lens[b], 0));
        all_see = __reduce_min_sync(0xFFFFFFFFu, all_see);
        for (; job < jobs; job += kLoadWarps) {
            const int n = job >> 2, stage = n % kStages;  // tile 2 j: keys, 2 j + 1: values of key tile j
            const int later = slot_of(job + 2 * kLoadWarps);
            const bool more = job + kLoadWarps < jobs;
            if (!warp_ready(&bars->empty[stage], (n / kStages & 1u) ^ 1u, abort_flag, status)) break;
            const unsigned votes = __ballot_sync(0xFFFFFFFFu, now >= 0);
            if (lane == 0 && !(n & 1)) *const_cast<volatile uint32_t*>(&bars->there[there_row(n >> 1)][job & 3]) = votes;
            const uint32_t dst = sKV + stage * kTile + (job & 3) * 32 * 128;
            const int tile = job >> 3;  // of this CTA
            const bool guard = (job & 4) && min(static_cast<int64_t>(tile0 + tile + 1) * kKeys, a.prefix) > all_see;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                copy_wait<1>();
                __syncwarp();
                if (guard) {
#pragma unroll 1
                    for (int i = h * kChunks / 2; i < (h + 1) * kChunks / 2; ++i)
                        if (take_nan(raw + 512 * i + 16 * lane)) atomicMin(&bars->lost_from, tile);
                }
#pragma unroll
                for (int i = h * kChunks / 2; i < (h + 1) * kChunks / 2; ++i) {
                    const uint4 u = ld_shared16(raw + 512 * i + 16 * lane);
                    // rows 8 apart have the same permutation
                    const int odd = kStep < 8 ? i & 1 : 0;
                    const uint32_t down = dst + 128 * kStep * (i - odd);
                    const uint32_t w[4] = {swap ? u.z : u.x, swap ? u.w : u.y, swap ? u.x : u.z, swap ? u.y : u.w};
                    st_shared16(down + at[odd][0], f16_lo(w[0]), f16_hi(w[0]), f16_lo(w[1]), f16_hi(w[1]));
                    st_shared16(down + at[odd][1], f16_lo(w[2]), f16_hi(w[2]), f16_lo(w[3]), f16_hi(w[3]));
                }
                __syncwarp();  // the codes are read: the next ones may come
                if (more) copy(job + kLoadWarps, next, h);
                else copy_commit();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->full[stage]);
            if (later >= 0) {
                const int far = job + 2 * kLoadWarps;
                const uint8_t* from = (far & 4 ? a.v_cache : a.k_cache) + static_cast<int64_t>(hk) * a.D;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(from + later * row_bytes) : "memory");
            }
            now = next;
            next = later;
        }
        copy_wait<0>();
      }
    }
    tc_fence_before();
    // The parts of the cluster's CTAs, added up in the order of the prefix:
    // each CTA does its share of the rows.  (Whatever happened above, every
    // thread comes by here: no CTA waits for one that gave up.)
    cluster_sync_all();
    if (warp < kMainWarps) {
        const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
        const int per = 2 * kRows / ctas;
        const uint32_t ml0 = smem_u32(bars->ml);
#pragma unroll 2
        for (int i = threadIdx.x; i < per * (DP / 4); i += 32 * kMainWarps) {
            const int r = rank * per + i / (DP / 4), ch = i % (DP / 4);
            const int x = r / kRows, row = r - x * kRows, tok = row / G;
            const uint32_t at = (x == 0 ? sQ : sKV) + 4 * DP * row + 16 * (ch ^ (row & 7));
            const int64_t b = b0 + x * tpt + tok;
            float2 ml[kMaxCluster];
            float4 v[kMaxCluster];
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {  // all of them on their way at once
                const int from = min(k, ctas - 1);
                ml[k] = ld_dsmem_v2(map_to_rank(ml0 + 8 * r, from));
                v[k] = ld_dsmem_v4(map_to_rank(at, from));
            }
            float top = -INFINITY, sum = 0.0f, o[4] = {};
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) top = k < ctas ? fmaxf(top, ml[k].x) : top;
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {
                // (an empty part has written nothing; a row whose scores are all NaN has no maximum, but a sum)
                if (k >= ctas || ml[k].y == 0.0f) continue;
                const float take = ex2(ml[k].x - top);
                sum += ml[k].y * take;
                o[0] += v[k].x * take, o[1] += v[k].y * take, o[2] += v[k].z * take, o[3] += v[k].w * take;
            }
            if (tok >= tpt || b >= a.B) continue;
            const int64_t to = ((static_cast<int64_t>(split / ctas) * a.Hkv + hk) * a.B + b) * G + (row - tok * G);
            *reinterpret_cast<float4*>(a.part_o + to * DP + 4 * ch) = make_float4(o[0], o[1], o[2], o[3]);
            if (ch == 0) a.part_ml[to] = make_float2(top, sum);
        }
    }
    cluster_sync_all();  // (nobody's memory goes while it is read)
    if (warp == kMainWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_attention_prefix(const DecodeArgs& a, const PrefixPlan& plan, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(plan.row_blocks * a.Hkv * plan.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = plan.dim == 64 ? smem_bytes<64>() : smem_bytes<128>();
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, plan.dim == 64 ? attention_prefix<64> : attention_prefix<128>, a, plan);
}

cudaError_t prepare_attention_prefix() {
    const cudaError_t e = cudaFuncSetAttribute(attention_prefix<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes<64>()));
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(attention_prefix<128>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem_bytes<128>()));
}

}  // namespace fp8k
