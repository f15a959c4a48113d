// scaled_api.cu -- the entry points of scored routing and of the float8 block-scaled operators
// (declared in include/moe.h): argument checks, workspace layouts and the choice of kernels.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>

#include "scaled.cuh"

namespace moe {

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Pointers that the kernels read or write as 4-byte words.
bool words(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned(p, 4)) return false;
    return true;
}

moe_status check_weights(const moe_scaled_weights *w) {
    if (!w || w->hidden <= 0 || w->ffn <= 0 || w->n_experts <= 0) return MOE_ERR_INVALID_ARG;
    if (w->hidden % 16 || w->ffn % 16 || (w->shared != 0 && w->shared != 1))
        return MOE_ERR_INVALID_ARG;
    if (w->n_experts > kMaxE || w->hidden > kScaledMaxDim || w->ffn > kScaledMaxDim)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// moe_scaled_set_wait_limit: these operators have no handle to keep it in.
std::atomic<uint64_t> g_wait_ns{2000000000ull};

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_scored(const float *d_logits, int T, int E, int k,
                            const moe_route_rule *host_rule, int32_t *d_ids, float *d_w,
                            int32_t *d_counts, int32_t *d_offsets, int32_t *d_perm,
                            int32_t *d_inv_perm, uint32_t *d_status, void *d_ws,
                            size_t ws_bytes, void *stream) {
    if (!d_logits || !host_rule || !d_ids || !d_w || !d_counts || !d_offsets || !d_perm || !d_ws)
        return MOE_ERR_INVALID_ARG;
    const moe_route_rule &r = *host_rule;
    if (T <= 0 || E <= 0 || k <= 0 || k > kMaxK || k > E) return MOE_ERR_INVALID_ARG;
    if (r.score != MOE_SCORE_SOFTMAX && r.score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (r.n_group <= 0 || r.n_group > 32 || E % r.n_group) return MOE_ERR_INVALID_ARG;
    const int per = E / r.n_group;
    if (r.topk_group <= 0 || r.topk_group > r.n_group || k > r.topk_group * per)
        return MOE_ERR_INVALID_ARG;
    if (r.group_top < 1 || r.group_top > 2 || r.group_top > per || !std::isfinite(r.scale))
        return MOE_ERR_INVALID_ARG;
    // pairs and the chunks of tokens are counted in 32 bits
    if (E > kMaxE || T > (1 << 30) || (int64_t)T * k > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (!words({d_logits, r.d_bias, d_ids, d_w, d_counts, d_offsets, d_perm, d_inv_perm, d_status}) ||
        !aligned(d_ws, 256))
        return MOE_ERR_ALIGNMENT;
    size_t need = 0;
    if (moe_route_workspace_size(T, E, k, &need) != MOE_OK) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    return launch_route_scored(d_logits, T, E, k, r, d_ids, d_w, d_counts, d_offsets, d_perm,
                               d_inv_perm, d_status, d_ws,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status moe_scaled_quantize(const void *d_x, int dtype, int T, int K, int64_t ldx,
                               uint8_t *d_q, int64_t ldq, float *d_s, int64_t lds,
                               uint32_t *d_status, void *stream) {
    if (!dtype_ok(dtype) || T < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!d_x || !d_q || !d_s)) return MOE_ERR_INVALID_ARG;   // empty tensors have no address
    if (ldx < K || ldq < K || lds < T) return MOE_ERR_INVALID_ARG;
    if (!aligned(d_x, dtype_bytes(dtype)) || !aligned(d_q, 16) || ldq % 16 ||
        !words({d_s, d_status}))
        return MOE_ERR_ALIGNMENT;
    // a warp per four rows and block, counted in 32 bits, as rows and columns are
    if (T > (1 << 30) || K > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    if (((int64_t)T + 3) / 4 * sblocks(K) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    return launch_scaled_quantize(d_x, dtype, T, K, ldx, d_q, ldq, d_s, lds, d_status,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status moe_scaled_matmul_workspace_size(int M, int N, int K, size_t *bytes) {
    if (!bytes || M < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    *bytes = scaled_matmul_ws_bytes(M, N, K);
    return MOE_OK;
}

moe_status moe_scaled_matmul(const uint8_t *d_a, int64_t lda, const float *d_as, int64_t ldas,
                             int M, int K, const uint8_t *d_b, int64_t ldb, const float *d_bs,
                             int N, void *d_out, int dtype, int64_t ldo, uint32_t *d_status,
                             void *d_ws, size_t ws_bytes, void *stream) {
    if (!d_b || !d_bs || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (M > 0 && (!d_a || !d_as || !d_out)) return MOE_ERR_INVALID_ARG;
    if (M < 0 || N <= 0 || K <= 0 || lda < K || ldb < K || ldas < M || ldo < N)
        return MOE_ERR_INVALID_ARG;
    // the kernels' tile counts and coordinates are 32-bit
    if (N > (1 << 30) || M > (1 << 30) || K > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    if (lda >= (int64_t(1) << 40) || ldb >= (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
    if (!aligned(d_a, 16) || !aligned(d_b, 16) || lda % 16 || ldb % 16 ||
        !aligned(d_out, dtype_bytes(dtype)) || !words({d_as, d_bs, d_status}) ||
        !aligned(d_ws, 256))
        return MOE_ERR_ALIGNMENT;
    const size_t need = scaled_matmul_ws_bytes(M, N, K);
    if (need && (!d_ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    if (M == 0) return MOE_OK;
    const ScaledMatmulArgs a{d_a, lda, d_as, ldas, M, K, d_b, ldb, d_bs, N, d_out, dtype, ldo,
                             d_status, g_wait_ns.load(std::memory_order_relaxed)};
    return launch_scaled_matmul(a, d_ws, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status moe_scaled_experts_workspace_size(const moe_scaled_weights *host_weights,
                                             int max_tokens, int k, size_t *bytes) {
    const moe_status st = check_weights(host_weights);
    if (st != MOE_OK) return st;
    if (!bytes || max_tokens <= 0 || k <= 0 || k > kMaxK || k > host_weights->n_experts)
        return MOE_ERR_INVALID_ARG;
    if ((int64_t)max_tokens * (k + 1) > kScaledMaxSlots) return MOE_ERR_UNSUPPORTED;
    // the small-batch kernels' workspace can exceed that of a slightly larger batch
    *bytes = std::max(scaled_experts_ws_bytes(*host_weights, max_tokens, k),
                      scaled_experts_ws_bytes(*host_weights, std::min(max_tokens, kSmallExpertsT), k));
    return MOE_OK;
}

moe_status moe_scaled_experts(const moe_scaled_weights *host_weights, const void *d_x,
                              int x_dtype, int T, int k, const int32_t *d_ids, const float *d_w,
                              const int32_t *d_offsets, const int32_t *d_inv_perm,
                              const float *d_gate, void *d_out, int out_dtype, uint32_t *d_status, void *d_ws, size_t ws_bytes,
                              void *stream) {
    const moe_status st = check_weights(host_weights);
    if (st != MOE_OK) return st;
    const moe_scaled_weights &w = *host_weights;
    if (!w.d_gate || !w.d_up || !w.d_down || !w.d_gate_s || !w.d_up_s || !w.d_down_s)
        return MOE_ERR_INVALID_ARG;
    if (!d_x || !d_ids || !d_w || !d_offsets || !d_inv_perm || !d_out || !d_ws)
        return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype) || (d_gate && !w.shared))
        return MOE_ERR_INVALID_ARG;
    if (T <= 0 || k <= 0 || k > kMaxK || k > w.n_experts) return MOE_ERR_INVALID_ARG;
    if ((int64_t)T * (k + 1) > kScaledMaxSlots) return MOE_ERR_UNSUPPORTED;
    if (!aligned(w.d_gate, 16) || !aligned(w.d_up, 16) || !aligned(w.d_down, 16) ||
        !aligned(d_x, 16) || !aligned(d_out, 16) || !aligned(d_ws, 256) ||
        !words({w.d_gate_s, w.d_up_s, w.d_down_s, d_ids, d_w, d_offsets, d_inv_perm,
                d_gate, d_status}))
        return MOE_ERR_ALIGNMENT;
    if (ws_bytes < scaled_experts_ws_bytes(w, T, k)) return MOE_ERR_WORKSPACE;
    ScaledExpertsArgs a{};
    a.w = w;
    a.x = d_x;
    a.x_dt = x_dtype;
    a.T = T;
    a.k = k;
    a.ids = d_ids;
    a.rw = d_w;
    a.offsets = d_offsets;
    a.inv_perm = d_inv_perm;
    a.gate = d_gate;
    a.out = d_out;
    a.out_dt = out_dtype;
    a.status = d_status;
    a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    return launch_scaled_experts(a, d_ws, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status moe_scaled_set_wait_limit(uint64_t ns) {
    if (ns == 0) return MOE_ERR_INVALID_ARG;
    g_wait_ns.store(ns, std::memory_order_relaxed);
    return MOE_OK;
}

}  // extern "C"
