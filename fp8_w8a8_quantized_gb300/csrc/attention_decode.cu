// Attention of one new token per request over the paged FP8 cache:
//   out[b, h] = v_scale sum_j w_j v_j / sum_j w_j,
//   w_j = 2^(y_j - m + 7),  y_j = scale log2(e) k_scale q . k_j   (7: kLift)
// in one pass over the cached tokens with the running maximum m, the running
// sum l and the running output o of the softmax (as in attention_prompt.cu: m
// follows the maximum in steps of at least 2^8).
//
// Bound by reading the cache: 2 D bytes a token and key head, each used for
// the G = Hq / Hkv queries of the group.  A warp takes 32 tokens of one key
// head at a time.  Asynchronous copies bring them into a ring of its own in
// shared memory (no barrier but the warp's own), kStages steps deep: up to 192
// KB of loads in flight an SM.
//
//   S^T [16 tokens x 8 queries] = K [16 x D] Q^T     m16n8k16, f16, fp32 sums
//   O^T [D x 8 queries]        += V^T [D x 16] P^T
//
// E4M3 codes convert to f16 exactly.  The sums over D and over tokens do not
// care in which order their terms come, so the fragments' index k stands for
// whatever makes a lane's loads 16 bytes wide: in S, lane (g, t) reads bytes
// 16 t .. 16 t + 15 of tokens g and g + 8; in O it reads bytes 16 g .. 16 g +
// 15 of tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9, and the bytes of two tokens are
// interleaved with a byte permute before they are converted.  A query is
// taken as f16 after its exponent is taken out (exact to 2^-38 of its largest
// element); P is f16.
//
// The tokens of all requests are one line of work, cut evenly among the CTAs
// by the lengths on the device: each CTA sums them up itself.  What a CTA
// holds of a request whose tokens it has alone goes to `out`, the rest as (m,
// l, o) to the workspace, from where attention_decode_join adds it up, in the
// order of the tokens.
//
// Measured, heads of 128: 64 requests of 257 to 16001 tokens, 64 / 8 heads, 510
// MB in 87 us: 3 us to the first copy and 5 until it is there, some 70 at 7.1 to
// 7.4 TB/s, 8 between the first CTA's end and the last's (more copies in flight
// make that worse, not better: a ring that runs on into the next request 93 us,
// one that is refilled a step earlier 96), 5 for the joining kernel.  One request
// of 16383 tokens, 32 / 8 heads: 13.9 us, of which 5 are bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "attention_tile.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

constexpr int kTile = 32;            // tokens of a warp's step
constexpr int kWarps = 8;            // warps of a CTA
constexpr int kCtas = 152;           // CTAs at most (one per SM)
constexpr int64_t kMaxPlan = 4096;   // requests up to which the work is cut by tokens
constexpr int kBatch = 4;            // parts of a row that are loaded at a time
constexpr int kWholeSteps = 4;       // steps of a request that one CTA does as a whole
// What a CTA could have read in the time that it takes to end one request and to
// get into the next, some 2.5 us (64 requests of 257 to 16001 tokens: 88.8 us;
// without it the CTAs with three requests end 8 us after those with one, 92.2).
// Alone, a request has nothing to be balanced against.
constexpr int kEntryBytes = 128 * 1024;
constexpr int kMinTokens = 64;       // tokens of a request that are worth a CTA

// A request whose steps several CTAs share, for the kernel that joins them.
struct Cut {
    int64_t first, end;  // its steps, counted over all requests
    int64_t per;         // steps of a CTA (0: the request is not cut)
    int32_t request, group;
};

struct Shape {
    int heads;   // key heads of a CTA at a time (a warp has one)
    int ways;    // warps that share a head's tokens
    int groups;  // (blocks of key heads) x (blocks of query rows)
    int blocks;  // blocks of query rows of a key head
};

template <int NT, int W>
__host__ __device__ inline Shape shape_of(int Hq, int Hkv) {
    Shape s;
    s.heads = Hkv < W ? Hkv : W;
    s.ways = W / s.heads;
    s.blocks = (Hq / Hkv + 8 * NT - 1) / (8 * NT);
    s.groups = (Hkv + s.heads - 1) / s.heads * s.blocks;
    return s;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint2 ld_shared8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// Steps of a CTA: an even share, and no fewer than are worth a CTA.  (32-bit
// division where the numbers allow: the 64-bit one takes a microsecond here.)
__device__ __forceinline__ int64_t divide_up(int64_t n, int64_t d) {
    n += d - 1;
    return (n | d) >> 32 ? n / d : static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
}

// The partial results in the workspace: after the cuts, (m, l) and then o of
// [cta][0: the request that the CTA begins in, 1: the one it ends in][head][row].
struct Parts {
    Cut* cuts;
    float2* ml;
    float* o;
};
template <int NT, int DP, int W>
__host__ __device__ inline size_t parts_rows(int heads) {
    return static_cast<size_t>(kCtas) * 2 * heads * 8 * NT;
}
template <int NT, int DP, int W>
__device__ __forceinline__ Parts parts_of(void* ws, int heads) {
    Parts p;
    p.cuts = static_cast<Cut*>(ws);
    p.ml = reinterpret_cast<float2*>(p.cuts + kCtas);
    p.o = reinterpret_cast<float*>(p.ml + parts_rows<NT, DP, W>(heads));
    return p;
}

// A warp's ring: kStages steps of kTile tokens' keys, then values, in rows of DP
// bytes.  16-byte chunk c of row r lies at c ^ key_swizzle(r) (values:
// value_swizzle(r)), so that the fragments' 16-byte reads meet no bank twice.
template <int DP>
struct Ring {
    static constexpr int kStages = DP == 128 ? 3 : 6;
    static constexpr uint32_t kHalf = kTile * DP;       // bytes of the keys of a step
    static constexpr uint32_t kBytes = 2 * kHalf * kStages;
    static constexpr int kChunks = DP / 16;
    __device__ static uint32_t key(int r, int c) {
        return static_cast<uint32_t>(r * DP + 16 * (DP == 128 ? c ^ ((r & 1) << 2) : c));
    }
    __device__ static uint32_t value(int r, int c) {
        return static_cast<uint32_t>(r * DP + 16 * (c ^ (DP == 128 ? (r >> 1 & 3) << 1 : r >> 1 & 3)));
    }
};

// NT: tiles of 8 queries.  DP: 64 or 128, at least D.  W: warps of a CTA.
template <int NT, int DP, int W>
__global__ void __launch_bounds__(W * 32, 1) attention_decode(const DecodeArgs a, const bool planned) {
    using R16 = Ring<DP>;
    constexpr int R = 8 * NT;
    constexpr int MT = DP / 16;  // tiles of 16 output elements
    constexpr int ST = R16::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    int64_t* upto = reinterpret_cast<int64_t*>(smem + W * R16::kBytes);  // [B + 1] steps before request b
    __shared__ int64_t warp_sums[W];
    __shared__ uint32_t there_of[W][ST];  // which tokens of a step exist
    const int warp = threadIdx.x >> 5, lane = lane_id();
    const int g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait_primary();

    const Shape sh = shape_of<NT, W>(a.Hq, a.Hkv);
    const int G = a.Hq / a.Hkv;
    const int64_t room = a.width * a.page;
    const int step = kTile * sh.ways;
    const int entry = a.B > 1 ? kEntryBytes / (2 * DP * kTile * W) : 0;
    // (tokens before `skip` are the prefix kernel's)
    auto length = [&](int64_t b) {
        const int64_t n = a.lens[b] < room ? a.lens[b] : room;
        return n > a.skip ? n - a.skip : int64_t(0);
    };

    // the line of work
    int64_t per = 0, lo, hi;
    if (planned) {
        // (a request without tokens has one step: someone has to write its zeros;
        // the first `entry` steps of each stand for the time that it takes to get into it)
        auto upto_lane = [&](int64_t b) {
            int64_t x = b < a.B ? max(divide_up(length(b), step), int64_t(1)) + entry : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                if (lane >= d) x += y;
            }
            return x;
        };
        int64_t carry = 0;
        if (a.B <= 32) {  // each warp for itself, all with the same values: nobody waits
            const int64_t x = upto_lane(lane);
            if (lane < a.B) upto[lane + 1] = x;
            if (lane == 0) upto[0] = 0;
            __syncwarp();
        }
        for (int64_t b0 = 0; a.B > 32 && b0 < a.B; b0 += W * 32) {
            const int64_t b = b0 + threadIdx.x;
            int64_t x = upto_lane(b);
            if (lane == 31) warp_sums[warp] = x;
            __syncthreads();
            int64_t before = carry;
            for (int w = 0; w < W; ++w) {
                if (w == warp) x += before;
                before += warp_sums[w];
            }
            carry = before;
            if (b < a.B) upto[b + 1] = x;
            __syncthreads();
        }
        if (a.B > 32) {
            if (threadIdx.x == 0) upto[0] = 0;
            __syncthreads();
        }
        const int64_t total = upto[a.B] * sh.groups;
        per = max(divide_up(total, gridDim.x), int64_t(max(kMinTokens / step, 1)));
        lo = min(per * blockIdx.x, total);
        hi = min(lo + per, total);
    } else {  // so many requests that each goes to one CTA as a whole
        lo = blockIdx.x;
        hi = a.B * sh.groups;
    }
    const Parts parts = parts_of<NT, DP, W>(a.workspace, sh.heads);
    const bool by_request = a.B * sh.groups <= kCtas;  // the cuts' order: requests, or CTAs that begin in one
    if (planned && threadIdx.x == 0 && !by_request) parts.cuts[blockIdx.x].per = 0;

    const int way = warp / sh.heads, my_head = warp - way * sh.heads;
    const bool works = way < sh.ways;
    const uint32_t ring = smem_u32(smem) + warp * R16::kBytes;
    const int64_t begin = lo;
    while (lo < hi) {
        // the request that step `lo` lies in, and how far this CTA goes in it
        int64_t b, first, end, inside;  // its steps on the line, and how many are before this CTA's
        int u0, u1;                     // this CTA's steps of tokens
        int group = 0;
        if (planned) {
            int64_t at = lo;
            while (at >= upto[a.B]) {
                at -= upto[a.B];
                ++group;
            }
            int x = 0, y = static_cast<int>(a.B);
            while (y - x > 1) {
                const int mid = (x + y) >> 1;
                if (upto[mid] <= at) x = mid; else y = mid;
            }
            b = x;
            first = lo - at + upto[b];
            end = lo - at + upto[b + 1];
            inside = lo - first;
            u0 = static_cast<int>(max(inside - entry, int64_t(0)));
            u1 = static_cast<int>(max(min(end, hi) - first - entry, int64_t(0)));
            // the CTA that begins a request, or that begins inside one, tells of the cut
            if (threadIdx.x == 0 && (by_request ? inside == 0 : inside > 0 && inside <= per)) {
                const bool cut = by_request ? hi < end : true;
                parts.cuts[by_request ? group * a.B + b : blockIdx.x] =
                    Cut{first, end, cut ? per : 0, static_cast<int32_t>(b), group};
            }
        } else {
            group = static_cast<int>(lo / a.B);
            b = lo - group * a.B;
            first = end = inside = u0 = 0;
            u1 = static_cast<int>(divide_up(length(b), step));
        }
        const bool whole = !planned || (lo == first && hi >= end);
        const int slot = lo == begin ? 0 : 1;  // (only a CTA's first and last request can be cut)
        lo = planned ? min(end, hi) : lo + gridDim.x;

        const int64_t len = length(b);
        const int hk = group / sh.blocks * sh.heads + my_head;
        const int r0 = group % sh.blocks * R;
        const bool on = works && hk < a.Hkv;

        float o[MT][NT][4];
        float m[NT][2], l[NT][2], c[NT][2];
        uint32_t q[NT][DP / 16][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][x][e] = 0.0f;
            m[x][0] = m[x][1] = -INFINITY;
            l[x][0] = l[x][1] = 0.0f;
        }
        if (on) {
            const float unit = a.scale * kLog2e * a.k_scale[hk * a.scale_stride];
            uint4 u[NT][DP / 64][2];  // the queries, on their way while the first tokens are
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) {
                    const int row = r0 + 8 * x + g, d = 64 * j + 16 * t;
                    u[x][j][0] = u[x][j][1] = make_uint4(0, 0, 0, 0);
                    if (row < G && d < a.D) {
                        const uint4* src = reinterpret_cast<const uint4*>(
                            a.q + b * a.ldq + static_cast<int64_t>(hk * G + row) * a.D + d);
                        u[x][j][0] = src[0];
                        u[x][j][1] = src[1];
                    }
                }
            const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * a.D;
            const uint8_t* kc = a.k_cache + static_cast<int64_t>(hk) * a.D;
            const uint8_t* vc = a.v_cache + static_cast<int64_t>(hk) * a.D;
            const int32_t* own_row = a.table + b * a.ld_table;
            const unsigned page = static_cast<unsigned>(a.page);
            // the slot of a lane's token of a step; -1 where there is none
            auto slot_of = [&](int u) {
                const int64_t tok = a.skip + (static_cast<int64_t>(u) * sh.ways + way) * kTile + lane;
                if (u >= u1 || tok - a.skip >= len) return -1;
                const unsigned pg = static_cast<unsigned>(tok) / page;
                const int id = (tok < a.prefix ? a.table : own_row)[pg];
                if (id < 0 || id >= a.n_pages) return -1;
                return static_cast<int>(id * page + (static_cast<unsigned>(tok) - pg * page));
            };
            auto issue = [&](int stage, int slots) {
                const unsigned votes = __ballot_sync(0xFFFFFFFFu, slots >= 0);
                if (lane == 0) there_of[warp][stage] = votes;
                const uint32_t dst = ring + stage * 2 * R16::kHalf;
#pragma unroll
                for (int i = 0; i < kTile * R16::kChunks / 32; ++i) {
                    const int r = (32 * i + lane) / R16::kChunks, ch = lane % R16::kChunks;
                    const int s = __shfl_sync(0xFFFFFFFFu, slots, r);
                    const bool there = s >= 0 && 16 * ch < a.D;
                    const int64_t off = s * row_bytes + 16 * ch;
                    copy_async16(dst + R16::key(r, ch), kc + off, there);
                    copy_async16(dst + R16::kHalf + R16::value(r, ch), vc + off, there);
                }
            };
            int ahead[ST];  // the slots of the next steps to be issued
#pragma unroll
            for (int i = 0; i < ST; ++i) ahead[i] = slot_of(u0 + i);
#pragma unroll
            for (int i = 0; i < ST - 1; ++i) {
                if (u0 + i < u1) issue(i, ahead[i]);
                copy_commit();
            }
            int next = ahead[ST - 1];
            if (a.splits > 0 && inside == 0 && way == 0) {
                // what the prefix kernel has of this request
                const int64_t stride = static_cast<int64_t>(a.Hkv) * a.B * G;
                const int64_t at0 = static_cast<int64_t>(hk) * a.B * G + b * G + r0;
                for (int i0 = 0; i0 < a.splits; i0 += kBatch) {
                    float2 ml[NT][2][kBatch];
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) {
                                const int row = 8 * x + 2 * t + e;
                                ml[x][e][i] = make_float2(-INFINITY, 0.0f);
                                if (r0 + row < G && i0 + i < a.splits)
                                    ml[x][e][i] = a.part_ml[at0 + row + (i0 + i) * stride];
                            }
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 8 * x + 2 * t + e;
                            if (r0 + row >= G) continue;
                            const float* src = a.part_o + (at0 + row + i0 * stride) * DP + DP / 8 * g;
                            float4 v[kBatch][MT / 2];
#pragma unroll
                            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                                for (int y = 0; y < MT / 2; ++y)
                                    v[i][y] = i0 + i < a.splits
                                                  ? reinterpret_cast<const float4*>(src + i * stride * DP)[y]
                                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            float top = m[x][e];
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[x][e][i].x);
                            const float keep = m[x][e] == -INFINITY ? 0.0f : ex2(m[x][e] - top);
                            m[x][e] = top;
                            l[x][e] *= keep;
#pragma unroll
                            for (int y = 0; y < MT; ++y) {
                                o[y][x][e] *= keep;
                                o[y][x][e + 2] *= keep;
                            }
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) {
                                const float take = ml[x][e][i].x == -INFINITY ? 0.0f : ex2(ml[x][e][i].x - top);
                                if (g == 0) l[x][e] += ml[x][e][i].y * take;  // (summed over the lanes in the end)
#pragma unroll
                                for (int y = 0; y < MT / 2; ++y) {
                                    o[2 * y][x][e] += v[i][y].x * take;
                                    o[2 * y][x][e + 2] += v[i][y].y * take;
                                    o[2 * y + 1][x][e] += v[i][y].z * take;
                                    o[2 * y + 1][x][e + 2] += v[i][y].w * take;
                                }
                            }
                        }
                }
            }


            // queries: row g of each tile, the elements that this lane's keys meet
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) top = top_of(u[x][j][1], top_of(u[x][j][0], top));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int shift = query_shift(top);
#pragma unroll
                for (int j = 0; j < DP / 64; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t w[4] = {u[x][j][e].x, u[x][j][e].y, u[x][j][e].z, u[x][j][e].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // elements 8 e + 2 i, + 1 of the 16: step 4 j + (4 e + i) / 2
                            const uint32_t h = pack_f16(scaled(bf16lo(w[i]), shift),
                                                        scaled(bf16hi(w[i]), shift));
                            q[x][4 * j + (4 * e + i) / 2][i & 1] = h;
                        }
                    }
                const float mine = scaled(unit, -shift);
                c[x][0] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t);
                c[x][1] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t + 4);
            }

            int stage = 0;
            for (int u = u0; u < u1; ++u) {
                copy_wait<ST - 2>();
                __syncwarp();  // step u has landed for all lanes, and all are done with step u - 1
                const unsigned there = there_of[warp][stage];
                const uint32_t src = ring + stage * 2 * R16::kHalf;
                if (u + ST - 1 < u1) issue(stage == 0 ? ST - 1 : stage - 1, next);
                copy_commit();
                next = slot_of(u + ST);
                stage = stage + 1 == ST ? 0 : stage + 1;

                float s[2][NT][4];  // of 16 tokens each
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[h][y][e] = 0.0f;
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 k0 = ld_shared16(src + R16::key(16 * h + g, 4 * j + t));
                        const uint4 k1 = ld_shared16(src + R16::key(16 * h + g + 8, 4 * j + t));
                        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w};
                        const uint32_t w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a0 = f16_lo(w0[i]), a1 = f16_lo(w1[i]);
                            const uint32_t a2 = f16_hi(w0[i]), a3 = f16_hi(w1[i]);
#pragma unroll
                            for (int y = 0; y < NT; ++y)
                                mma_16816(s[h][y], a0, a1, a2, a3, q[y][4 * j + i][0], q[y][4 * j + i][1]);
                        }
                    }
                }
                // softmax: columns 2 t, 2 t + 1 of tokens 16 h + g and 16 h + g + 8
                bool raise = false;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[h][y][e] *= c[y][e & 1];
                            if (!((there >> (16 * h + 8 * (e >> 1) + g)) & 1u)) s[h][y][e] = -INFINITY;
                            raise |= s[h][y][e] - m[y][e & 1] > kSlack;
                        }
                if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = fmaxf(fmaxf(s[0][y][e], s[0][y][e + 2]), fmaxf(s[1][y][e], s[1][y][e + 2]));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                            if (top - m[y][e] > kSlack) {
                                const float keep = m[y][e] == -INFINITY ? 0.0f : ex2(m[y][e] - top);
                                m[y][e] = top;
                                l[y][e] *= keep;
#pragma unroll
                                for (int i = 0; i < MT; ++i) {
                                    o[i][y][e] *= keep;
                                    o[i][y][e + 2] *= keep;
                                }
                            }
                        }
                }
                uint32_t p[2][NT][2];
#pragma unroll
                for (int y = 0; y < NT; ++y) {
                    const float b0 = m[y][0] == -INFINITY ? 0.0f : m[y][0] - kLift;
                    const float b1 = m[y][1] == -INFINITY ? 0.0f : m[y][1] - kLift;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[h][y][e] = ex2(s[h][y][e] - (e & 1 ? b1 : b0));
                            l[y][e & 1] += s[h][y][e];
                        }
                        p[h][y][0] = transpose_8x8(pack_f16(s[h][y][0], s[h][y][1]));
                        p[h][y][1] = transpose_8x8(pack_f16(s[h][y][2], s[h][y][3]));
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[4][DP / 32];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 16 * h + 2 * t + (r & 1) + 8 * (r >> 1);
                        const uint32_t half = src + R16::kHalf;
                        if constexpr (DP == 128) {
                            const uint4 w = ld_shared16(half + R16::value(row, g));
                            v[r][0] = w.x, v[r][1] = w.y, v[r][2] = w.z, v[r][3] = w.w;
                        } else {
                            const uint2 w = ld_shared8(half + R16::value(row, g >> 1) + 8 * (g & 1));
                            v[r][0] = w.x, v[r][1] = w.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < DP / 32; ++i) {
                        const uint32_t p0 = __byte_perm(v[0][i], v[1][i], 0x5140);
                        const uint32_t p1 = __byte_perm(v[0][i], v[1][i], 0x7362);
                        const uint32_t p2 = __byte_perm(v[2][i], v[3][i], 0x5140);
                        const uint32_t p3 = __byte_perm(v[2][i], v[3][i], 0x7362);
                        const uint32_t a0 = f16_lo(p0), a1 = f16_hi(p0), a2 = f16_lo(p2), a3 = f16_hi(p2);
                        const uint32_t c0 = f16_lo(p1), c1 = f16_hi(p1), c2 = f16_lo(p3), c3 = f16_hi(p3);
#pragma unroll
                        for (int y = 0; y < NT; ++y) {
                            mma_16816(o[2 * i][y], a0, a1, a2, a3, p[h][y][0], p[h][y][1]);
                            mma_16816(o[2 * i + 1][y], c0, c1, c2, c3, p[h][y][0], p[h][y][1]);
                        }
                    }
                }
            }
            copy_wait<0>();
            __syncwarp();
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        l[y][e] += __shfl_xor_sync(0xFFFFFFFFu, l[y][e], d);
        }

        // Several warps with one head: added up in shared memory, each row by
        // the warps of its head in turn.
        if (sh.ways > 1) {
            float* so = reinterpret_cast<float*>(smem);  // (where the rings were)
            float2* sml = reinterpret_cast<float2*>(so + W * R * DP);
            __syncthreads();
            if (on && way > 0) {
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * y + 2 * t + e;
                        float* dst = so + (warp * R + row) * DP + DP / 8 * g;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            dst[2 * i] = o[i][y][e];
                            dst[2 * i + 1] = o[i][y][e + 2];
                        }
                        if (g == 0) sml[warp * R + row] = make_float2(m[y][e], l[y][e]);
                    }
            }
            __syncthreads();
            if (on && way == 0) {
                for (int w = 1; w < sh.ways; ++w) {
                    const int from = w * sh.heads + my_head;
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 8 * y + 2 * t + e;
                            const float2 ml = sml[from * R + row];
                            const float top = fmaxf(m[y][e], ml.x);
                            const float keep = m[y][e] == -INFINITY ? 0.0f : ex2(m[y][e] - top);
                            const float take = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
                            const float* src = so + (from * R + row) * DP + DP / 8 * g;
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                o[i][y][e] = o[i][y][e] * keep + src[2 * i] * take;
                                o[i][y][e + 2] = o[i][y][e + 2] * keep + src[2 * i + 1] * take;
                            }
                            m[y][e] = top;
                            l[y][e] = l[y][e] * keep + ml.y * take;
                        }
                }
            }
        }
        if (sh.ways > 1 && lo < hi) __syncthreads();  // before the rings fill again
        if (!on || way > 0) continue;
        if (whole) {
            const float vs = a.v_scale[hk * a.scale_stride];
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = r0 + 8 * y + 2 * t + e;
                    const float inv = l[y][e] == 0.0f ? 0.0f : vs / l[y][e];
                    const int d = DP / 8 * g;
                    if (row < G && d < a.D) {
                        uint16_t* dst = a.out + b * a.ldo + static_cast<int64_t>(hk * G + row) * a.D + d;
                        uint32_t w[MT];
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const __nv_bfloat162 v =
                                __floats2bfloat162_rn(o[i][y][e] * inv, o[i][y][e + 2] * inv);
                            w[i] = *reinterpret_cast<const uint32_t*>(&v);
                        }
#pragma unroll
                        for (int i = 0; i < MT; i += 4)
                            *reinterpret_cast<uint4*>(dst + 2 * i) =
                                make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                    }
                }
        } else {
            const size_t at = ((static_cast<size_t>(blockIdx.x) * 2 + slot) * sh.heads + my_head) * R;
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * y + 2 * t + e;
                    float* dst = parts.o + (at + row) * DP + DP / 8 * g;
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(
                            o[i][y][e], o[i][y][e + 2], o[i + 1][y][e], o[i + 1][y][e + 2]);
                    if (g == 0) parts.ml[at + row] = make_float2(m[y][e], l[y][e]);
                }
        }
    }
}

// Adds up the parts of the requests that several CTAs hold: the CTAs (x, ...)
// do the request of cut x.  A row of few parts is a warp's; the parts of a
// row that has many are dealt to the CTA's warps, whose sums are then added in
// the warps' order.
//
// JW: warps of a CTA.  16 where a row is a CTA's (one request of 16383 tokens,
// 128 parts a row, one round of loads: 13.9 us with the kernel before it; with 8
// warps 16.4), 8 where it is a warp's (64 ragged requests 88.1 us instead of 88.9:
// 16 warps of 90 registers have an SM to themselves, and half of them no row).
constexpr int kJoinBatch = 8;  // parts on their way
template <int NT, int DP, int W, int JW>
__global__ void __launch_bounds__(JW * 32) attention_decode_join(const DecodeArgs a) {
    constexpr int R = 8 * NT;
    constexpr int V = DP / 32;
    __shared__ float s_o[JW][DP];
    __shared__ float2 s_ml[JW];
    pdl_launch_dependents();
    pdl_wait_primary();
    const Shape sh = shape_of<NT, W>(a.Hq, a.Hkv);
    const Parts parts = parts_of<NT, DP, W>(a.workspace, sh.heads);
    const Cut cut = parts.cuts[blockIdx.x];
    if (cut.per == 0) return;
    const int c0 = static_cast<int>(divide_up(cut.first + 1, cut.per) - 1);
    const bool begins = cut.per * c0 == cut.first;  // else c0 has its part in slot 1
    const int last = static_cast<int>(divide_up(cut.end, cut.per) - 1);
    const int G = a.Hq / a.Hkv, lane = lane_id(), warp = threadIdx.x >> 5;
    const int r0 = cut.group % sh.blocks * R, h0 = cut.group / sh.blocks * sh.heads;
    const int rows = min(R, G - r0), items = rows * min(sh.heads, a.Hkv - h0);
    const bool few = last - c0 < 2 * kJoinBatch;
    const int step = few ? 1 : JW, offset = few ? 0 : warp;
    for (int y = few ? blockIdx.y * JW + warp : blockIdx.y; y < items;
         y += few ? gridDim.y * JW : gridDim.y) {
        const int head = y / rows, row = y - head * rows;
        float m = -INFINITY, l = 0.0f, o[V] = {};
        for (int cta = c0 + offset; cta <= last; cta += kJoinBatch * step) {
            float2 ml[kJoinBatch];
            float part[kJoinBatch][V];
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                const int from = cta + i * step;
                ml[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int e = 0; e < V; ++e) part[i][e] = 0.0f;
                if (from <= last) {
                    const int slot = from == c0 && !begins ? 1 : 0;
                    const size_t at = ((static_cast<size_t>(from) * 2 + slot) * sh.heads + head) * R + row;
                    ml[i] = parts.ml[at];
#pragma unroll
                    for (int e = 0; e < V; ++e) part[i][e] = parts.o[at * DP + 32 * e + lane];
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) top = fmaxf(top, ml[i].x);
            const float keep = m == -INFINITY ? 0.0f : ex2(m - top);
            m = top;
            l *= keep;
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] *= keep;
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                const float take = ml[i].x == -INFINITY ? 0.0f : ex2(ml[i].x - top);
                l += ml[i].y * take;
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] += part[i][e] * take;
            }
        }
        const int hk = h0 + head;
        const float vs = a.v_scale[hk * a.scale_stride];
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + cut.request * a.ldo +
                             static_cast<int64_t>(hk * G + r0 + row) * a.D;
        if (few) {
            const float inv = l == 0.0f ? 0.0f : vs / l;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (32 * e + lane < a.D) dst[32 * e + lane] = __float2bfloat16_rn(o[e] * inv);
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) s_o[warp][32 * e + lane] = o[e];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (threadIdx.x < DP) {
            float top = -INFINITY;
            for (int w = 0; w < JW; ++w) top = fmaxf(top, s_ml[w].x);
            float sum = 0.0f, all = 0.0f;
            for (int w = 0; w < JW; ++w) {
                const float take = s_ml[w].x == -INFINITY ? 0.0f : ex2(s_ml[w].x - top);
                sum += s_o[w][threadIdx.x] * take;
                all += s_ml[w].y * take;
            }
            const float inv = all == 0.0f ? 0.0f : vs / all;
            if (static_cast<int>(threadIdx.x) < a.D) dst[threadIdx.x] = __float2bfloat16_rn(sum * inv);
        }
    }
}

template <int NT, int DP>
struct Launch {
    static constexpr int W = kWarps;
    static size_t smem(int64_t B) {
        return W * Ring<DP>::kBytes + (B <= kMaxPlan ? (B + 1) * 8 : 0);
    }
    static size_t workspace(int64_t B, int Hq, int Hkv) {
        if (B > kMaxPlan) return 0;
        const Shape s = shape_of<NT, W>(Hq, Hkv);
        return sizeof(Cut) * kCtas + parts_rows<NT, DP, W>(s.heads) * (sizeof(float2) + DP * sizeof(float));
    }
    static cudaError_t prepare() {
        return cudaFuncSetAttribute(attention_decode<NT, DP, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(smem(kMaxPlan)));
    }
    static cudaError_t run(const DecodeArgs& a, cudaStream_t st) {
        const Shape s = shape_of<NT, W>(a.Hq, a.Hkv);
        // Contexts of a few steps at most are not cut either: a second launch to
        // join their parts takes longer than the steps do (7 requests of up to
        // 301 tokens, 2 key heads: 6.2 us whole, 7.8 us cut and joined).
        const int64_t steps = (a.width * a.page - a.skip + kTile * s.ways - 1) / (kTile * s.ways);
        const bool planned = a.B <= kMaxPlan && steps > kWholeSteps;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        const int ctas = a.num_sms < kCtas ? a.num_sms : kCtas;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(W * 32);
        cfg.dynamicSmemBytes = smem(a.B);
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, attention_decode<NT, DP, W>, a, planned);
        if (e != cudaSuccess || !planned || ctas < 2) return e;
        // Few requests have many parts each: a CTA for every row.  Many have a
        // few each, most of them, but one may still have almost all.
        const int64_t cuts = a.B * s.groups <= kCtas ? a.B * s.groups : ctas;
        const int64_t rows = s.heads * (a.Hq / a.Hkv < 8 * NT ? a.Hq / a.Hkv : 8 * NT);
        cfg.dynamicSmemBytes = 0;
        if (cuts <= 16) {
            cfg.gridDim = dim3(static_cast<unsigned>(cuts), static_cast<unsigned>(rows));
            cfg.blockDim = dim3(16 * 32);
            return cudaLaunchKernelEx(&cfg, attention_decode_join<NT, DP, W, 16>, a);
        }
        cfg.gridDim = dim3(static_cast<unsigned>(cuts), static_cast<unsigned>((rows + 7) / 8));
        cfg.blockDim = dim3(8 * 32);
        return cudaLaunchKernelEx(&cfg, attention_decode_join<NT, DP, W, 8>, a);
    }
};

using Narrow64 = Launch<1, 64>;
using Narrow128 = Launch<1, 128>;
using Wide64 = Launch<2, 64>;
using Wide128 = Launch<2, 128>;

}  // namespace

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix) {
    const int q = static_cast<int>(Hq), kv = static_cast<int>(Hkv);
    const size_t own = Hq / Hkv <= 8
                           ? (D <= 64 ? Narrow64::workspace(B, q, kv) : Narrow128::workspace(B, q, kv))
                           : (D <= 64 ? Wide64::workspace(B, q, kv) : Wide128::workspace(B, q, kv));
    const PrefixPlan p = prefix_plan(B, Hq, Hkv, D, prefix);
    return (own + 255) / 256 * 256 + p.parts_bytes();
}

cudaError_t launch_attention_decode(const DecodeArgs& given, cudaStream_t st) {
    DecodeArgs a = given;
    const PrefixPlan p = prefix_plan(a.B, a.Hq, a.Hkv, a.D, a.prefix);
    a.skip = 0;
    a.splits = p.parts();
    if (p.splits > 0) {
        a.skip = a.prefix;
        const size_t all = attention_decode_workspace(a.B, a.Hq, a.Hkv, a.D, a.prefix);
        a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + all - p.parts_bytes());
        a.part_ml = reinterpret_cast<float2*>(a.part_o + p.rows() * p.dim);
        const cudaError_t e = launch_attention_prefix(a, p, st);
        if (e != cudaSuccess) return e;
    }
    if (a.Hq / a.Hkv <= 8) return a.D <= 64 ? Narrow64::run(a, st) : Narrow128::run(a, st);
    return a.D <= 64 ? Wide64::run(a, st) : Wide128::run(a, st);
}

cudaError_t prepare_attention_decode() {
    for (cudaError_t e : {Narrow64::prepare(), Narrow128::prepare(), Wide64::prepare(), Wide128::prepare()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace fp8k
