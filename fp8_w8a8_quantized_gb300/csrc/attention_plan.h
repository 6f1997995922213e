// Host arithmetic of the shared-prefix kernel (attention_prefix.cu), apart from
// it so that it can be checked without a GPU: how the prefix is cut into parts,
// and which place of a CTA's rings a key tile takes.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define FP8K_BOTH __host__ __device__
#else
#define FP8K_BOTH
#endif

namespace fp8k {

constexpr int kRows = 128;  // rows of a query tile
constexpr int kKeys = 128;  // keys of a tile

// The keys of key tile j and then its values take the next stages of one ring.
constexpr int kPrefixStages = 4;
FP8K_BOTH constexpr uint32_t key_stage(uint32_t j) { return 2 * j % kPrefixStages; }
FP8K_BOTH constexpr uint32_t value_stage(uint32_t j) { return (2 * j + 1) % kPrefixStages; }

// Where the words that say which tokens of key tile j exist lie.  Softmax warps
// read them, and no barrier of the key ring waits for those: a stage is free for
// key tile j + 2 when the MMAs of S have read key tile j.  The keys of tile j + 4
// wait for S of tile j + 2, which is issued behind P of tile j + 1, which each
// softmax warp writes after it has read the words of tile j.
constexpr int kThereRows = 4;
FP8K_BOTH constexpr uint32_t there_row(uint32_t j) { return j % kThereRows; }

constexpr int kMaxCluster = 4;  // (clusters of 8 found room for fewer CTAs: 71 us instead of 47)
constexpr int kFillSms = 152;   // CTAs that the parts should come to

// The tokens that all requests share, read once for all.
struct PrefixPlan {
    int splits;          // parts of the prefix (0: not worth it, the decode kernel reads it)
    int cluster;         // CTAs of a cluster: parts that are added up before they are written
    int tiles;           // key tiles of a part
    int dim;             // D rounded up to 64 or 128
    int64_t row_blocks;  // blocks of query rows
    int64_t all_rows;    // B * Hq
    int parts() const { return splits ? splits / cluster : 0; }
    int64_t rows() const { return parts() * all_rows; }
    size_t parts_bytes() const { return static_cast<size_t>(rows()) * (dim * 4 + 8); }
};

inline PrefixPlan prefix_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix) {
    PrefixPlan p = {};
    p.dim = D <= 64 ? 64 : 128;
    p.all_rows = B * Hq;
    if (B < 2 || prefix < kKeys) return p;
    const int64_t tpt = kRows / (Hq / Hkv);
    p.row_blocks = (B + 2 * tpt - 1) / (2 * tpt);
    const int64_t tiles = (prefix + kKeys - 1) / kKeys, items = p.row_blocks * Hkv;
    int64_t splits = items >= kFillSms ? 1 : kFillSms / items;
    if (splits > tiles) splits = tiles;
    p.cluster = splits >= kMaxCluster ? kMaxCluster : splits >= 2 ? 2 : 1;
    splits = splits / p.cluster * p.cluster;
    p.tiles = static_cast<int>((tiles + splits - 1) / splits);
    // Worth it where it is faster than the decode kernel on the same tokens, by
    // what both were measured to need (page size 16, 300 tokens beside the
    // prefix): that one reads B times the prefix, out of L2 mostly, at 8.6
    // bytes/ps with 8 heads of 128, 5 with heads of 64; this one costs 18 us
    // and 2.4 us a key tile of a CTA.  The call at 32/8 heads of 128, own reading
    // against this: B = 16, 8192 tokens 42 / 30 us, 2048 tokens 19 / 25; B = 64,
    // 2048 tokens 44 / 32, 512 tokens 23 / 31; B = 4, 32768 tokens 39 / 50.
    const double own_us = static_cast<double>(B) * prefix * 2 * Hkv * D / (D > 64 ? 8.6e6 : 5.0e6);
    if (own_us < 18.0 + 2.4 * p.tiles) {
        p.tiles = 0;
        return p;
    }
    // whole clusters (the last parts may be empty), and no empty ones
    const int64_t used = (tiles + p.tiles - 1) / p.tiles;
    p.splits = static_cast<int>((used + p.cluster - 1) / p.cluster * p.cluster);
    return p;
}

}  // namespace fp8k
