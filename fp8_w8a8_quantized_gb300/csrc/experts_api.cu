// C-ABI entry points of the expert block (fp8w8a8.h): host-side argument checks
// and the launches of moe_route.cu, quant.cu, gemm_grouped.cu and
// residual_norm.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "fp8w8a8.h"
#include "launch.h"

namespace {

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 38;  // elements between two rows
constexpr int64_t kMost = int64_t(1) << 30;   // rows and widths that the kernels count in 32 bits
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTop = 32;
constexpr int64_t kMaxTokens = int64_t(1) << 23;  // of a routing (counts of its parts in 16 bits)
constexpr int64_t kMaxNormWidth = 32768;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool aligned(std::initializer_list<const void*> ps, uintptr_t a) {
    for (const void* p : ps)
        if (!aligned(p, a)) return false;
    return true;
}

bool any_out(std::initializer_list<int64_t> sizes, int64_t most = kMax31) {
    for (int64_t n : sizes)
        if (n < 0 || n > most) return true;
    return false;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// A bf16 matrix of K columns with leading dimension ld.
fp8_status_t check_rows(const void* p, int64_t ld, int64_t K) {
    if (!p || ld < K || ld > kMaxLd) return FP8_ERR_INVALID_ARG;
    return ld % 8 || !aligned(p, 16) ? FP8_ERR_UNSUPPORTED : FP8_OK;
}

fp8_status_t check_grouped_sizes(int64_t E, int64_t R, int64_t N, int64_t K, bool swiglu) {
    if (any_out({E, R, N, K}) || E < 1 || (swiglu && N % 2)) return FP8_ERR_INVALID_ARG;
    if (K == 0 || K % 16 || E > kMaxExperts || N > kMost / E || K > kMost || R > kMost)
        return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status_t check_grouped(const uint8_t* wq, const float* s_w, const int32_t* offsets,
                           const void* y) {
    if (!wq || !s_w || !offsets || !y) return FP8_ERR_INVALID_ARG;
    return aligned({wq, y}, 16) && aligned({s_w, offsets}, 4) ? FP8_OK : FP8_ERR_UNSUPPORTED;
}

fp8_status_t said(cudaError_t e) { return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

fp8k::GroupedArgs grouped_args(const uint8_t* xq, const float* s_tok, const uint8_t* wq,
                               const float* s_w, const int32_t* offsets, int64_t E, int64_t R,
                               int64_t N, int64_t K, int swiglu, void* y, void* workspace,
                               bool zeroed) {
    fp8k::GroupedArgs a;
    a.xq = xq;
    a.s_tok = s_tok;
    a.wq = wq;
    a.s_w = s_w;
    a.offsets = offsets;
    a.E = static_cast<int>(E), a.R = static_cast<int>(R);
    a.N = static_cast<int>(N), a.K = static_cast<int>(K);
    a.swiglu = swiglu != 0;
    a.y = y;
    a.workspace = workspace;
    a.zeroed = zeroed;
    return a;
}

}  // namespace

extern "C" {

size_t fp8_moe_route_workspace_size(int64_t T, int64_t E, int64_t top_k) {
    if (T < 0 || E < 1 || E > kMaxExperts || top_k < 1 || top_k > E || top_k > kMaxTop ||
        T > kMaxTokens)
        return 0;
    return fp8k::moe_route_workspace(T, E, top_k);
}

fp8_status_t fp8_moe_route(const void* logits, int logits_fp32, int64_t ld, int64_t T, int64_t E,
                           int64_t top_k, int renormalize, float scale, int32_t* expert_ids,
                           float* weights, int32_t* offsets, int32_t* row_token,
                           int32_t* token_row, void* workspace, size_t ws_bytes, void* stream) {
    if (any_out({T, E, top_k}) || top_k < 1 || top_k > E || !std::isfinite(scale))
        return FP8_ERR_INVALID_ARG;
    if (E > kMaxExperts || top_k > kMaxTop || T > kMaxTokens) return FP8_ERR_UNSUPPORTED;
    if (!offsets || (T > 0 && (!logits || !expert_ids || !weights || !row_token || !token_row)))
        return FP8_ERR_INVALID_ARG;
    if (T > 0 && (ld < E || ld > kMaxLd)) return FP8_ERR_INVALID_ARG;
    if (!aligned(logits, logits_fp32 ? 4 : 2) ||
        !aligned({expert_ids, weights, offsets, row_token, token_row}, 4))
        return FP8_ERR_UNSUPPORTED;
    const size_t need = fp8k::moe_route_workspace(T, E, top_k);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 16)))
        return FP8_ERR_WORKSPACE;
    int num_sms = 0;
    unsigned* status = nullptr;
    const fp8_status_t st = fp8k::device_info(&num_sms, &status);
    if (st != FP8_OK) return st;
    fp8k::RouteArgs a;
    a.logits = logits;
    a.fp32 = logits_fp32 != 0;
    a.ld = ld, a.T = T;
    a.E = static_cast<int>(E), a.k = static_cast<int>(top_k);
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.ids = expert_ids;
    a.weights = weights;
    a.offsets = offsets, a.row_token = row_token, a.token_row = token_row;
    a.workspace = static_cast<uint16_t*>(workspace);
    return said(fp8k::launch_moe_route(a, as_stream(stream)));
}

size_t fp8_grouped_gemm_workspace_size(int64_t E, int64_t R, int64_t N, int64_t K) {
    if (check_grouped_sizes(E, R, N, K, false) != FP8_OK || R == 0 || N == 0) return 0;
    return fp8k::gemm_grouped_workspace(E, R, N, K);
}

fp8_status_t fp8_grouped_gemm(const uint8_t* xq, const float* s_tok, const uint8_t* wq,
                              const float* s_w, const int32_t* offsets, int64_t E, int64_t R,
                              int64_t N, int64_t K, int swiglu, void* y_bf16, void* workspace,
                              size_t ws_bytes, void* stream) {
    fp8_status_t st = check_grouped_sizes(E, R, N, K, swiglu != 0);
    if (st != FP8_OK || R == 0 || N == 0) return st;
    if (!xq || !s_tok) return FP8_ERR_INVALID_ARG;
    if (!aligned(xq, 16) || !aligned(s_tok, 4)) return FP8_ERR_UNSUPPORTED;
    if ((st = check_grouped(wq, s_w, offsets, y_bf16)) != FP8_OK) return st;
    const size_t need = fp8k::gemm_grouped_workspace(E, R, N, K);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return FP8_ERR_WORKSPACE;
    fp8k::GroupedArgs a =
        grouped_args(xq, s_tok, wq, s_w, offsets, E, R, N, K, swiglu, y_bf16, workspace, false);
    if ((st = fp8k::device_info(&a.num_sms, &a.status, &a.pair_clusters)) != FP8_OK) return st;
    return said(fp8k::launch_gemm_grouped(a, as_stream(stream)));
}

// [codes R * K | scales 4 * R | the product's workspace], each at a multiple of 256
size_t fp8_grouped_linear_workspace_size(int64_t E, int64_t R, int64_t N, int64_t K) {
    if (check_grouped_sizes(E, R, N, K, false) != FP8_OK || R == 0 || N == 0) return 0;
    return round256(static_cast<size_t>(R) * static_cast<size_t>(K)) +
           round256(4 * static_cast<size_t>(R)) + fp8k::gemm_grouped_workspace(E, R, N, K);
}

fp8_status_t fp8_grouped_linear(const void* x_bf16, int64_t T, int64_t ldx,
                                const int32_t* row_token, const uint8_t* wq, const float* s_w,
                                const int32_t* offsets, int64_t E, int64_t R, int64_t N, int64_t K,
                                int swiglu, void* y_bf16, void* workspace, size_t ws_bytes,
                                void* stream) {
    fp8_status_t st = check_grouped_sizes(E, R, N, K, swiglu != 0);
    if (st != FP8_OK) return st;
    if (any_out({T}) || (!row_token && T != R)) return FP8_ERR_INVALID_ARG;
    if (R == 0 || N == 0) return FP8_OK;
    if (T > 0 && (st = check_rows(x_bf16, ldx, K)) != FP8_OK) return st;
    if (!aligned(row_token, 4)) return FP8_ERR_UNSUPPORTED;
    if ((st = check_grouped(wq, s_w, offsets, y_bf16)) != FP8_OK) return st;
    const size_t need = fp8_grouped_linear_workspace_size(E, R, N, K);
    if (!workspace || ws_bytes < need || !aligned(workspace, 256)) return FP8_ERR_WORKSPACE;
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* scales = xq + round256(static_cast<size_t>(R) * static_cast<size_t>(K));
    uint8_t* rest = scales + round256(4 * static_cast<size_t>(R));
    float* s_tok = reinterpret_cast<float*>(scales);
    fp8k::GroupedArgs a =
        grouped_args(xq, s_tok, wq, s_w, offsets, E, R, N, K, swiglu, y_bf16, rest, true);
    if ((st = fp8k::device_info(&a.num_sms, &a.status, &a.pair_clusters)) != FP8_OK) return st;
    const cudaError_t e = fp8k::launch_quant_gather(
        x_bf16, T, R, K, ldx, row_token, xq, s_tok, reinterpret_cast<uint32_t*>(rest),
        fp8k::gemm_grouped_zero_words(), as_stream(stream));
    return e != cudaSuccess ? FP8_ERR_CUDA
                            : said(fp8k::launch_gemm_grouped(a, as_stream(stream)));
}

fp8_status_t fp8_residual_norm_quant(const void* h, int64_t ldh, const void* y, int64_t ldy,
                                     int64_t R, const int32_t* token_row, const float* weights,
                                     int64_t top_k, const void* gamma_post, const void* gate,
                                     int64_t ldg, const void* gamma, float eps,
                                     float residual_scale, float branch_scale, int64_t T,
                                     int64_t K, void* h_out, int64_t ldho, void* z_out,
                                     uint8_t* xq, int64_t ldq, float* s_tok, void* stream) {
    if (any_out({T, R, K, top_k})) return FP8_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(residual_scale) ||
        !std::isfinite(branch_scale))
        return FP8_ERR_INVALID_ARG;
    if (top_k == 0 && R != T) return FP8_ERR_INVALID_ARG;
    if (K == 0 || K % 16 || K > kMaxNormWidth || top_k > kMaxTop) return FP8_ERR_UNSUPPORTED;
    if (T == 0) return FP8_OK;
    if ((top_k > 0 && !token_row) || (xq == nullptr) != (s_tok == nullptr) ||
        ((z_out || xq) && !gamma))
        return FP8_ERR_INVALID_ARG;
    fp8_status_t st = FP8_OK;
    if ((st = check_rows(h, ldh, K)) != FP8_OK || (st = check_rows(h_out, ldho, K)) != FP8_OK ||
        (R > 0 && (st = check_rows(y, ldy, K)) != FP8_OK) ||
        (gate && ldg != 0 && (st = check_rows(gate, ldg, K)) != FP8_OK))
        return st;
    if (xq && (ldq < K || ldq > kMaxLd)) return FP8_ERR_INVALID_ARG;
    if (!aligned({gamma_post, gate, gamma, z_out, xq}, 16) ||
        !aligned({token_row, weights, s_tok}, 4) || (xq && ldq % 16))
        return FP8_ERR_UNSUPPORTED;
    int num_sms = 0;
    unsigned* status = nullptr;
    if ((st = fp8k::device_info(&num_sms, &status)) != FP8_OK) return st;
    fp8k::ResidualNormArgs a;
    a.h = static_cast<const uint16_t*>(h), a.y = static_cast<const uint16_t*>(y);
    a.ldh = ldh, a.ldy = ldy, a.R = R;
    a.token_row = token_row;
    a.weights = weights;
    a.k = static_cast<int>(top_k);
    a.gamma_post = static_cast<const uint16_t*>(gamma_post);
    a.gate = static_cast<const uint16_t*>(gate);
    a.gamma = static_cast<const uint16_t*>(gamma);
    a.ldg = ldg;
    a.eps = eps, a.residual_scale = residual_scale, a.branch_scale = branch_scale;
    a.T = T, a.K = K;
    a.h_out = static_cast<uint16_t*>(h_out);
    a.ldho = ldho;
    a.z = static_cast<uint16_t*>(z_out);
    a.q = xq;
    a.ldq = ldq;
    a.s = s_tok;
    return said(fp8k::launch_residual_norm(a, as_stream(stream)));
}

}  // extern "C"
