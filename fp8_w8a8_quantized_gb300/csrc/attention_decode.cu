// Attention of one new token per request over the paged FP8 cache:
//   out[b, h] = v_scale sum_j w_j v_j / sum_j w_j,
//   w_j = 2^(y_j - m),  y_j = scale log2(e) k_scale q . k_j
// in one pass over the cached tokens with the running maximum m, the running
// sum l and the running output o of the softmax (as in attention_prompt.cu: m
// follows the maximum in steps of at least 2^8).
//
// Bound by reading the cache: 2 D bytes a token and key head, each used for
// the G = Hq / Hkv queries of the group, so nothing of it goes through shared
// memory or is read twice.  A warp takes 16 tokens of one key head at a time,
// straight from global memory into registers, the next 16 while it computes:
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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "launch.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8k {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;       // log2 of how far p may exceed 1 before m moves
constexpr int kTile = 16;            // tokens of a warp's step
constexpr int kCtas = 152;           // CTAs at most (one per SM)
constexpr int64_t kMaxPlan = 4096;   // requests up to which the work is cut by tokens
constexpr int kMinUnits = 4;         // steps that are worth a CTA

// Where the work of CTA `c` begins inside a request: that request's steps.
struct Cut {
    int64_t first, end;  // its steps, counted over all requests
    int64_t total;       // steps of all requests (a header's total of 0: no cut here)
    int32_t request, group;
    int32_t ctas, pad;
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Two E4M3 codes (low or high half of u) -> two f16 values, exact.
__device__ __forceinline__ uint32_t f16_lo(uint32_t u) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(r)
        : "r"(u));
    return r;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t u) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(u));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^n, for n beyond fp32's exponents too (as two factors).
__device__ __forceinline__ float scaled(float x, int n) {
    const int h = n / 2;
    return x * __uint_as_float(static_cast<uint32_t>(127 + h) << 23) *
           __uint_as_float(static_cast<uint32_t>(127 + n - h) << 23);
}

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_stream8(const uint8_t* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ int64_t cut_at(int64_t total, int c, int ctas) {
    return total / ctas * c + total % ctas * c / ctas;
}

// The partial results in the workspace: after kCtas cuts, (m, l) and then o of
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

// One request's tokens, as far as a warp is concerned.
template <int DP>
struct Tokens {
    static constexpr int KW = DP / 64;   // 16-byte loads of a token's keys
    static constexpr int VW = DP / 32;   // words of a lane's share of a token's values
    uint4 k[2][KW];
    uint32_t v[4][VW];
};

// NT: tiles of 8 queries.  DP: 64 or 128, at least D.  W: warps of a CTA.
template <int NT, int DP, int W>
__global__ void __launch_bounds__(W * 32, 1) attention_decode(const DecodeArgs a, const bool planned) {
    using Tok = Tokens<DP>;
    constexpr int R = 8 * NT;
    constexpr int MT = DP / 16;  // tiles of 16 output elements
    extern __shared__ __align__(16) uint8_t smem[];
    int64_t* upto = reinterpret_cast<int64_t*>(smem);      // [B + 1] steps before request b
    __shared__ int64_t warp_sums[W];
    const int warp = threadIdx.x >> 5, lane = lane_id();
    const int g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait_primary();

    const Shape sh = shape_of<NT, W>(a.Hq, a.Hkv);
    const int G = a.Hq / a.Hkv;
    const int64_t room = a.width * a.page;
    const int step = kTile * sh.ways;
    auto length = [&](int64_t b) {
        const int64_t n = a.lens[b];
        return n < 0 ? int64_t(0) : n < room ? n : room;
    };

    // the line of work
    int64_t total = 0, lo, hi;
    int ctas = gridDim.x;
    if (planned) {
        int64_t carry = 0;
        for (int64_t b0 = 0; b0 < a.B; b0 += W * 32) {
            const int64_t b = b0 + threadIdx.x;
            // (a request without tokens has one step: someone has to write its zeros)
            const int64_t n = b < a.B ? max((length(b) + step - 1) / step, int64_t(1)) : 0;
            int64_t x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                if (lane >= d) x += y;
            }
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
        if (threadIdx.x == 0) upto[0] = 0;
        __syncthreads();
        total = upto[a.B] * sh.groups;
        const int64_t worth = (total + kMinUnits - 1) / kMinUnits;
        ctas = worth < ctas ? static_cast<int>(worth) : ctas;
        lo = hi = 0;
        if (static_cast<int>(blockIdx.x) < ctas) {
            lo = cut_at(total, blockIdx.x, ctas);
            hi = cut_at(total, blockIdx.x + 1, ctas);
        }
    } else {  // so many requests that each goes to one CTA as a whole
        lo = blockIdx.x;
        hi = a.B * sh.groups;
    }
    const Parts parts = parts_of<NT, DP, W>(a.workspace, sh.heads);
    if (planned && threadIdx.x == 0 && static_cast<int>(blockIdx.x) >= ctas)
        parts.cuts[blockIdx.x].total = 0;

    const int way = warp / sh.heads, my_head = warp - way * sh.heads;
    const bool works = way < sh.ways;
    const int64_t begin = lo;
    while (lo < hi) {
        // the request that step `lo` lies in, and how far this CTA goes in it
        int64_t b, first, end, u0, u1;  // its steps; this CTA's, counted from its first
        int group;
        if (planned) {
            group = static_cast<int>(lo / upto[a.B]);
            const int64_t at = lo - group * upto[a.B];
            int64_t x = 0, y = a.B;
            while (y - x > 1) {
                const int64_t mid = (x + y) >> 1;
                if (upto[mid] <= at) x = mid; else y = mid;
            }
            b = x;
            first = group * upto[a.B] + upto[b];
            end = group * upto[a.B] + upto[b + 1];
            u0 = lo - first;
            u1 = min(end, hi) - first;
            if (lo == begin && threadIdx.x == 0) {
                Cut cut;
                cut.first = first;
                cut.end = end;
                cut.total = u0 > 0 ? total : 0;
                cut.request = static_cast<int32_t>(b);
                cut.group = group;
                cut.ctas = ctas;
                cut.pad = 0;
                parts.cuts[blockIdx.x] = cut;
            }
        } else {
            group = static_cast<int>(lo / a.B);
            b = lo - group * a.B;
            first = end = u0 = 0;
            u1 = (length(b) + step - 1) / step;
        }
        const bool whole = !planned || (lo == first && hi >= end);
        const int slot = lo == begin ? 0 : 1;  // (only a CTA's first and last request can be cut)
        lo = planned ? first + u1 : lo + gridDim.x;

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
            // queries: row g of each tile, the elements that this lane's keys meet
            const float unit = a.scale * kLog2e * a.k_scale[hk * a.scale_stride];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const int row = r0 + 8 * x + g;
                uint4 u[DP / 64][2];
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) {
                    u[j][0] = u[j][1] = make_uint4(0, 0, 0, 0);
                    const int d = 64 * j + 16 * t;
                    if (row < G && d < a.D) {
                        const uint4* src = reinterpret_cast<const uint4*>(
                            a.q + b * a.ldq + static_cast<int64_t>(hk * G + row) * a.D + d);
                        u[j][0] = src[0];
                        u[j][1] = src[1];
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t w[4] = {u[j][e].x, u[j][e].y, u[j][e].z, u[j][e].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
                    }
                }
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // the largest element goes to [2^14, 2^15)
                const int ex = top == 0 ? 14 : max(static_cast<int>(top >> 7), 1) - 127;
#pragma unroll
                for (int j = 0; j < DP / 64; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t w[4] = {u[j][e].x, u[j][e].y, u[j][e].z, u[j][e].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // elements 8 e + 2 i, + 1 of the 16: step 4 j + (4 e + i) / 2
                            const uint32_t h = pack_f16(scaled(bf16lo(w[i]), 14 - ex),
                                                        scaled(bf16hi(w[i]), 14 - ex));
                            q[x][4 * j + (4 * e + i) / 2][i & 1] = h;
                        }
                    }
                const float mine = scaled(unit, ex - 14);
                c[x][0] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t);
                c[x][1] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t + 4);
            }

            const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * a.D;
            const uint8_t* kc = a.k_cache + static_cast<int64_t>(hk) * a.D;
            const uint8_t* vc = a.v_cache + static_cast<int64_t>(hk) * a.D;
            const int32_t* own_row = a.table + b * a.ld_table;
            const int page = static_cast<int>(a.page);
            // the slot of token (lane mod 16) of a step, -1 where there is none
            auto slot_of = [&](int64_t u) {
                const int64_t tok = (u * sh.ways + way) * kTile + (lane & 15);
                if (u >= u1 || tok >= len) return -1;
                const int pg = static_cast<int>(tok) / page;
                const int id = __ldg((tok < a.prefix ? a.table : own_row) + pg);
                if (id < 0 || id >= a.n_pages) return -1;
                return id * page + (static_cast<int>(tok) - pg * page);
            };
            auto load_k = [&](Tok& x, int slots) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int s = __shfl_sync(0xFFFFFFFFu, slots, g + 8 * r);
#pragma unroll
                    for (int j = 0; j < Tok::KW; ++j) {
                        x.k[r][j] = make_uint4(0, 0, 0, 0);
                        const int d = 64 * j + 16 * t;
                        if (s >= 0 && d < a.D) x.k[r][j] = ld_stream(kc + s * row_bytes + d);
                    }
                }
            };
            auto load_v = [&](Tok& x, int slots) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int s = __shfl_sync(0xFFFFFFFFu, slots, 2 * t + (r & 1) + 8 * (r >> 1));
#pragma unroll
                    for (int i = 0; i < Tok::VW; ++i) x.v[r][i] = 0;
                    const int d = DP / 8 * g;
                    if (s >= 0 && d < a.D) {
                        const uint8_t* p = vc + s * row_bytes + d;
                        if constexpr (DP == 128) {
                            const uint4 w = ld_stream(p);
                            x.v[r][0] = w.x, x.v[r][1] = w.y, x.v[r][2] = w.z, x.v[r][3] = w.w;
                        } else {
                            const uint2 w = ld_stream8(p);
                            x.v[r][0] = w.x, x.v[r][1] = w.y;
                        }
                    }
                }
            };

            Tok x;
            int now = slot_of(u0);
            load_k(x, now);
            load_v(x, now);
            int next = slot_of(u0 + 1);
            for (int64_t u = u0; u < u1; ++u) {
                const unsigned there = __ballot_sync(0xFFFFFFFFu, now >= 0);
                const bool on0 = (there >> g) & 1u, on1 = (there >> (g + 8)) & 1u;
                float s[NT][4];
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[y][e] = 0.0f;
#pragma unroll
                for (int j = 0; j < Tok::KW; ++j) {
                    const uint32_t w0[4] = {x.k[0][j].x, x.k[0][j].y, x.k[0][j].z, x.k[0][j].w};
                    const uint32_t w1[4] = {x.k[1][j].x, x.k[1][j].y, x.k[1][j].z, x.k[1][j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = f16_lo(w0[i]), a1 = f16_lo(w1[i]);
                        const uint32_t a2 = f16_hi(w0[i]), a3 = f16_hi(w1[i]);
#pragma unroll
                        for (int y = 0; y < NT; ++y)
                            mma_16816(s[y], a0, a1, a2, a3, q[y][4 * j + i][0], q[y][4 * j + i][1]);
                    }
                }
                load_k(x, next);
                // softmax: columns 2 t, 2 t + 1 of tokens g and g + 8
                bool raise = false;
#pragma unroll
                for (int y = 0; y < NT; ++y) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[y][e] *= c[y][e & 1];
                        if (!(e < 2 ? on0 : on1)) s[y][e] = -INFINITY;
                        raise |= s[y][e] - m[y][e & 1] > kSlack;
                    }
                }
                if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = fmaxf(s[y][e], s[y][e + 2]);
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
                uint32_t p[NT][2];
#pragma unroll
                for (int y = 0; y < NT; ++y) {
                    const float b0 = m[y][0] == -INFINITY ? 0.0f : m[y][0];
                    const float b1 = m[y][1] == -INFINITY ? 0.0f : m[y][1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[y][e] = ex2(s[y][e] - (e & 1 ? b1 : b0));
                        l[y][e & 1] += s[y][e];
                    }
                    p[y][0] = transpose_8x8(pack_f16(s[y][0], s[y][1]));
                    p[y][1] = transpose_8x8(pack_f16(s[y][2], s[y][3]));
                }
#pragma unroll
                for (int i = 0; i < Tok::VW; ++i) {
                    const uint32_t p0 = __byte_perm(x.v[0][i], x.v[1][i], 0x5140);
                    const uint32_t p1 = __byte_perm(x.v[0][i], x.v[1][i], 0x7362);
                    const uint32_t p2 = __byte_perm(x.v[2][i], x.v[3][i], 0x5140);
                    const uint32_t p3 = __byte_perm(x.v[2][i], x.v[3][i], 0x7362);
                    const uint32_t a0 = f16_lo(p0), a1 = f16_hi(p0), a2 = f16_lo(p2), a3 = f16_hi(p2);
                    const uint32_t c0 = f16_lo(p1), c1 = f16_hi(p1), c2 = f16_lo(p3), c3 = f16_hi(p3);
#pragma unroll
                    for (int y = 0; y < NT; ++y) {
                        mma_16816(o[2 * i][y], a0, a1, a2, a3, p[y][0], p[y][1]);
                        mma_16816(o[2 * i + 1][y], c0, c1, c2, c3, p[y][0], p[y][1]);
                    }
                }
                load_v(x, next);
                now = next;
                next = slot_of(u + 2);
            }
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
            float* so = reinterpret_cast<float*>(smem + (planned ? (a.B + 1) * 8 + 8 : 0));
            so = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(so) + 15) & ~uintptr_t(15));
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

// Adds up the parts of a request that several CTAs hold.  CTA (c, y): the
// request in which CTA c begins, if c is the first one to begin inside it;
// rows y, y + gridDim.y, ... of its heads.  Each of the warps sums every
// kWarps-th part, then they are summed in their order.
constexpr int kJoinWarps = 8;
template <int NT, int DP, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_decode_join(const DecodeArgs a) {
    constexpr int R = 8 * NT;
    constexpr int V = DP / 32;
    __shared__ float s_o[kJoinWarps][DP];
    __shared__ float2 s_ml[kJoinWarps];
    pdl_launch_dependents();
    pdl_wait_primary();
    const Shape sh = shape_of<NT, W>(a.Hq, a.Hkv);
    const Parts parts = parts_of<NT, DP, W>(a.workspace, sh.heads);
    const int c1 = blockIdx.x + 1;
    const Cut cut = parts.cuts[c1];
    if (cut.total == 0) return;              // CTA c1 begins with a request's first token
    const int c0 = c1 - 1;
    const int64_t c0_from = cut_at(cut.total, c0, cut.ctas);
    if (c0_from > cut.first) return;         // an earlier CTA begins inside it too
    const bool begins = c0_from == cut.first;  // else c0 has its part in slot 1
    const int G = a.Hq / a.Hkv, lane = lane_id(), warp = threadIdx.x >> 5;
    int last = c1;
    while (last + 1 < cut.ctas && cut_at(cut.total, last + 1, cut.ctas) < cut.end) ++last;
    for (int y = blockIdx.y; y < sh.heads * R; y += gridDim.y) {
        const int head = y / R, row = y - head * R;
        const int hk = cut.group / sh.blocks * sh.heads + head;
        const int r = cut.group % sh.blocks * R + row;
        if (hk >= a.Hkv || r >= G) continue;
        auto at = [&](int cta) {
            const int slot = cta == c0 && !begins ? 1 : 0;
            return ((static_cast<size_t>(cta) * 2 + slot) * sh.heads + head) * R + row;
        };
        float m = -INFINITY, l = 0.0f, o[V] = {};
        for (int cta = c0 + warp; cta <= last; cta += kJoinWarps) {
            const size_t i = at(cta);
            const float2 ml = parts.ml[i];
            const float top = fmaxf(m, ml.x);
            const float keep = m == -INFINITY ? 0.0f : ex2(m - top);
            const float take = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = o[e] * keep + parts.o[i * DP + V * lane + e] * take;
            l = l * keep + ml.y * take;
            m = top;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) s_o[warp][V * lane + e] = o[e];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (threadIdx.x < DP) {
            float top = -INFINITY;
            for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w].x);
            float sum = 0.0f, all = 0.0f;
            for (int w = 0; w < kJoinWarps; ++w) {
                const float take = s_ml[w].x == -INFINITY ? 0.0f : ex2(s_ml[w].x - top);
                sum += s_o[w][threadIdx.x] * take;
                all += s_ml[w].y * take;
            }
            const float inv = all == 0.0f ? 0.0f : a.v_scale[hk * a.scale_stride] / all;
            if (static_cast<int>(threadIdx.x) < a.D)
                reinterpret_cast<__nv_bfloat16*>(a.out)[cut.request * a.ldo +
                                                        static_cast<int64_t>(hk * G + r) * a.D + threadIdx.x] =
                    __float2bfloat16_rn(sum * inv);
        }
    }
}

template <int NT, int DP, int W>
struct Launch {
    static size_t smem(int64_t B, int ways) {
        const size_t plan = B <= kMaxPlan ? (B + 1) * 8 + 24 : 16;
        return plan + (ways > 1 ? W * 8 * NT * (DP * 4 + 8) : 0);
    }
    static size_t workspace(int64_t B, int Hq, int Hkv) {
        if (B > kMaxPlan) return 0;
        const Shape s = shape_of<NT, W>(Hq, Hkv);
        return sizeof(Cut) * kCtas + parts_rows<NT, DP, W>(s.heads) * (sizeof(float2) + DP * sizeof(float));
    }
    static cudaError_t prepare() {
        return cudaFuncSetAttribute(attention_decode<NT, DP, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(smem(kMaxPlan, 2)));
    }
    static cudaError_t run(const DecodeArgs& a, cudaStream_t st) {
        const Shape s = shape_of<NT, W>(a.Hq, a.Hkv);
        const bool planned = a.B <= kMaxPlan;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        const int ctas = a.num_sms < kCtas ? a.num_sms : kCtas;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(W * 32);
        cfg.dynamicSmemBytes = smem(a.B, s.ways);
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, attention_decode<NT, DP, W>, a, planned);
        if (e != cudaSuccess || !planned || ctas < 2) return e;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), a.B <= 8 ? s.heads * 8 * NT : s.heads);
        cfg.blockDim = dim3(kJoinWarps * 32);
        cfg.dynamicSmemBytes = 0;
        return cudaLaunchKernelEx(&cfg, attention_decode_join<NT, DP, W>, a);
    }
};

using Narrow64 = Launch<1, 64, 16>;
using Narrow128 = Launch<1, 128, 16>;
using Wide64 = Launch<2, 64, 8>;
using Wide128 = Launch<2, 128, 8>;

}  // namespace

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t, int64_t) {
    const int q = static_cast<int>(Hq), kv = static_cast<int>(Hkv);
    if (Hq / Hkv <= 8) return D <= 64 ? Narrow64::workspace(B, q, kv) : Narrow128::workspace(B, q, kv);
    return D <= 64 ? Wide64::workspace(B, q, kv) : Wide128::workspace(B, q, kv);
}

cudaError_t launch_attention_decode(const DecodeArgs& a, cudaStream_t st) {
    if (a.Hq / a.Hkv <= 8) return a.D <= 64 ? Narrow64::run(a, st) : Narrow128::run(a, st);
    return a.D <= 64 ? Wide64::run(a, st) : Wide128::run(a, st);
}

cudaError_t prepare_attention_decode() {
    for (cudaError_t e : {Narrow64::prepare(), Narrow128::prepare(), Wide64::prepare(), Wide128::prepare()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace fp8k
