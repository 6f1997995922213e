// C-ABI entry points of the attention block (fp8w8a8.h): host-side argument
// checks and the launches of kv_slots.cu, norm_rope.cu, attention_prompt.cu and
// attention_decode.cu (with attention_prefix.cu).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "fp8w8a8.h"
#include "launch.h"

namespace {

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 38;  // elements between two tokens
constexpr int64_t kMaxGroup = 64;             // query heads per key head
constexpr int64_t kMaxAttentionDim = 128;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool any_out(std::initializer_list<int64_t> sizes, int64_t most = kMax31) {
    for (int64_t n : sizes)
        if (n < 0 || n > most) return true;
    return false;
}

// A [tokens, heads, D] bf16 tensor with token stride ld.
fp8_status_t check_tokens(const void* p, int64_t ld, int64_t heads, int64_t D) {
    if (!p || ld < heads * D || ld > kMaxLd) return FP8_ERR_INVALID_ARG;
    return ld % 8 || !aligned(p, 16) ? FP8_ERR_UNSUPPORTED : FP8_OK;
}

fp8_status_t check_heads(int64_t Hq, int64_t Hkv, int64_t D, float scale) {
    if (Hq < 1 || Hkv < 1 || D < 1 || Hq > kMax31 || Hkv > kMax31 || D > kMax31 || Hq % Hkv)
        return FP8_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return FP8_ERR_INVALID_ARG;
    if (D % 16 || D > kMaxAttentionDim || Hq / Hkv > kMaxGroup || Hkv > 65535)
        return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status_t said(cudaError_t e) { return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

fp8_status_t fp8_kv_slots(const int32_t* ctx_lens, const int32_t* new_lens, int64_t B,
                          const int32_t* free_pages, int64_t n_free, int64_t page_size,
                          int32_t* block_table, int64_t table_width, int64_t ld_table,
                          int64_t max_tokens, int64_t* slot_mapping, int32_t* positions,
                          int32_t* cu_seqlens, int32_t* seq_lens, int32_t* pages_used,
                          void* stream) {
    if (any_out({B, n_free, table_width, max_tokens, page_size}) || page_size < 1)
        return FP8_ERR_INVALID_ARG;
    if (!cu_seqlens || !pages_used || (B > 0 && (!ctx_lens || !new_lens || !seq_lens)) ||
        (n_free > 0 && !free_pages) || (max_tokens > 0 && (!slot_mapping || !positions)))
        return FP8_ERR_INVALID_ARG;
    if (B > 0 && table_width > 0 && (!block_table || ld_table < table_width || ld_table > kMaxLd))
        return FP8_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                          static_cast<const void*>(free_pages), static_cast<const void*>(block_table),
                          static_cast<const void*>(positions), static_cast<const void*>(cu_seqlens),
                          static_cast<const void*>(seq_lens), static_cast<const void*>(pages_used)})
        if (!aligned(p, 4)) return FP8_ERR_UNSUPPORTED;
    if (!aligned(slot_mapping, 8)) return FP8_ERR_UNSUPPORTED;
    int num_sms = 0;
    unsigned* status = nullptr;
    const fp8_status_t st = fp8k::device_info(&num_sms, &status);
    if (st != FP8_OK) return st;
    return said(fp8k::launch_kv_slots(ctx_lens, new_lens, B, free_pages, n_free, page_size,
                                      block_table, table_width, ld_table, max_tokens, slot_mapping,
                                      positions, cu_seqlens, seq_lens, pages_used, num_sms,
                                      as_stream(stream)));
}

fp8_status_t fp8_qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                              int64_t ldv, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                              const void* gamma_q, const void* gamma_k, float eps,
                              const int32_t* positions, const uint64_t* turns, int64_t rot_dim,
                              int interleaved, void* q_out, int64_t ldqo, void* k_out, int64_t ldko,
                              const float* k_scale, const float* v_scale, int64_t scale_stride,
                              const int64_t* slot_mapping, uint8_t* k_cache, uint8_t* v_cache,
                              int64_t n_slots, void* stream) {
    if (any_out({T, Hq, Hkv, D, rot_dim, n_slots}) || scale_stride < 0 || rot_dim > D)
        return FP8_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return FP8_ERR_INVALID_ARG;
    if (T == 0 || (Hq == 0 && Hkv == 0) || D == 0) return FP8_OK;
    if (D % 16 || D > 256 || rot_dim % 16 || Hq > 65536 || Hkv > 65536 || Hq + 2 * Hkv > 65536)
        return FP8_ERR_UNSUPPORTED;
    const bool cache = k_cache || v_cache;
    if (!positions || (rot_dim > 0 && !turns)) return FP8_ERR_INVALID_ARG;
    if (cache && (!k_cache || !v_cache || !k_scale || !v_scale)) return FP8_ERR_INVALID_ARG;
    if (!cache && Hkv > 0 && !k_out) return FP8_ERR_INVALID_ARG;
    fp8_status_t st = FP8_OK;
    if (Hq > 0 && ((st = check_tokens(q, ldq, Hq, D)) != FP8_OK ||
                   (st = check_tokens(q_out, ldqo, Hq, D)) != FP8_OK))
        return st;
    if (Hkv > 0 && ((st = check_tokens(k, ldk, Hkv, D)) != FP8_OK ||
                    (k_out && (st = check_tokens(k_out, ldko, Hkv, D)) != FP8_OK) ||
                    (cache && (st = check_tokens(v, ldv, Hkv, D)) != FP8_OK)))
        return st;
    if (!aligned(positions, 4) || !aligned(turns, 8) || !aligned(gamma_q, 16) ||
        !aligned(gamma_k, 16))
        return FP8_ERR_UNSUPPORTED;
    if (cache && (!aligned(k_cache, 8) || !aligned(v_cache, 8) || !aligned(k_scale, 4) ||
                  !aligned(v_scale, 4) || !aligned(slot_mapping, 8)))
        return FP8_ERR_UNSUPPORTED;
    int num_sms = 0;
    unsigned* status = nullptr;
    if ((st = fp8k::device_info(&num_sms, &status)) != FP8_OK) return st;
    fp8k::QkNormRopeArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.T = T;
    a.Hq = static_cast<int>(Hq), a.Hkv = static_cast<int>(Hkv), a.D = static_cast<int>(D);
    a.rot = static_cast<int>(rot_dim);
    a.pairs = interleaved != 0;
    a.gamma_q = static_cast<const uint16_t*>(gamma_q);
    a.gamma_k = static_cast<const uint16_t*>(gamma_k);
    a.eps = eps;
    a.positions = positions;
    a.turns = turns;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.k_out = static_cast<uint16_t*>(k_out);
    a.ldqo = ldqo, a.ldko = ldko;
    a.k_scale = k_scale, a.v_scale = v_scale;
    a.scale_stride = scale_stride;
    a.slot = slot_mapping;
    a.k_cache = k_cache, a.v_cache = v_cache;
    a.n_slots = n_slots;
    return said(fp8k::launch_qk_norm_rope(a, num_sms, as_stream(stream)));
}

fp8_status_t fp8_attention_prompt(const void* q, int64_t ldq, const void* k, int64_t ldk,
                                  const void* v, int64_t ldv, int64_t T, int64_t Hq, int64_t Hkv,
                                  int64_t D, const int32_t* cu_seqlens, int64_t S, float scale,
                                  void* out, int64_t ldo, void* stream) {
    if (any_out({T, S})) return FP8_ERR_INVALID_ARG;
    fp8_status_t st = check_heads(Hq, Hkv, D, scale);
    if (st != FP8_OK || T == 0 || S == 0) return st;
    if (!cu_seqlens) return FP8_ERR_INVALID_ARG;
    if ((st = check_tokens(q, ldq, Hq, D)) != FP8_OK ||
        (st = check_tokens(k, ldk, Hkv, D)) != FP8_OK ||
        (st = check_tokens(v, ldv, Hkv, D)) != FP8_OK ||
        (st = check_tokens(out, ldo, Hq, D)) != FP8_OK)
        return st;
    if (!aligned(cu_seqlens, 4) || T + S > kMax31 / Hkv) return FP8_ERR_UNSUPPORTED;
    fp8k::PromptArgs a;
    if ((st = fp8k::device_info(&a.num_sms, &a.status)) != FP8_OK) return st;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.T = T, a.B = S;
    a.cu = cu_seqlens;
    a.Hq = static_cast<int>(Hq), a.Hkv = static_cast<int>(Hkv), a.D = static_cast<int>(D);
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ldo = ldo;
    return said(fp8k::launch_attention_prompt(a, as_stream(stream)));
}

size_t fp8_attention_decode_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                                           int64_t table_width, int64_t page_size,
                                           int64_t prefix_len) {
    if (any_out({B, table_width, page_size, prefix_len}) || page_size < 1 ||
        table_width > kMax31 / page_size || prefix_len > table_width * page_size ||
        check_heads(Hq, Hkv, D, 1.0f) != FP8_OK || B * Hkv >= (int64_t(1) << 24) || B == 0)
        return 0;
    return fp8k::attention_decode_workspace(B, Hq, Hkv, D, prefix_len);
}

fp8_status_t fp8_attention_decode(const void* q, int64_t ldq, int64_t B, int64_t Hq, int64_t Hkv,
                                  int64_t D, const uint8_t* k_cache, const uint8_t* v_cache,
                                  int64_t n_slots, const float* k_scale, const float* v_scale,
                                  int64_t scale_stride, const int32_t* block_table,
                                  int64_t table_width, int64_t ld_table, int64_t page_size,
                                  const int32_t* seq_lens, int64_t prefix_len, float scale,
                                  void* out, int64_t ldo, void* workspace, size_t ws_bytes,
                                  void* stream) {
    if (any_out({B, n_slots, table_width, page_size, prefix_len}) || page_size < 1 ||
        scale_stride < 0)
        return FP8_ERR_INVALID_ARG;
    fp8_status_t st = check_heads(Hq, Hkv, D, scale);
    if (st != FP8_OK || B == 0) return st;
    if (table_width > kMax31 / page_size || B * Hkv >= (int64_t(1) << 24)) return FP8_ERR_UNSUPPORTED;
    if (prefix_len > table_width * page_size) return FP8_ERR_INVALID_ARG;
    if (!k_scale || !v_scale || !seq_lens) return FP8_ERR_INVALID_ARG;
    if (table_width > 0 && (!block_table || ld_table < table_width || ld_table > kMaxLd))
        return FP8_ERR_INVALID_ARG;
    if (n_slots >= page_size && table_width > 0 && (!k_cache || !v_cache))
        return FP8_ERR_INVALID_ARG;
    if ((st = check_tokens(q, ldq, Hq, D)) != FP8_OK ||
        (st = check_tokens(out, ldo, Hq, D)) != FP8_OK)
        return st;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return FP8_ERR_UNSUPPORTED;
    const size_t need = fp8k::attention_decode_workspace(B, Hq, Hkv, D, prefix_len);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return FP8_ERR_WORKSPACE;
    fp8k::DecodeArgs a;
    if ((st = fp8k::device_info(&a.num_sms, &a.status)) != FP8_OK) return st;
    a.q = static_cast<const uint16_t*>(q);
    a.ldq = ldq;
    a.B = B;
    a.Hq = static_cast<int>(Hq), a.Hkv = static_cast<int>(Hkv), a.D = static_cast<int>(D);
    a.k_cache = k_cache, a.v_cache = v_cache;
    a.n_pages = n_slots / page_size;
    a.k_scale = k_scale, a.v_scale = v_scale;
    a.scale_stride = scale_stride;
    a.table = block_table;
    a.width = table_width, a.ld_table = ld_table, a.page = page_size;
    a.lens = seq_lens;
    a.prefix = prefix_len;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ldo = ldo;
    a.workspace = workspace;
    return said(fp8k::launch_attention_decode(a, as_stream(stream)));
}

}  // extern "C"
