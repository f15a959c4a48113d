// k_scored.cu -- routing by scores: softmax or sigmoid of the logits, a balance bias that takes
// part in the choice alone, groups of experts of which the best stay, top-k, weights from the
// chosen scores.
//
// The order of the choice is that of 64-bit scores, so that a near-tie is decided as the formula
// decides it, whatever the order of a sum or the last bits of an fp32 exponential would say.
#include <math.h>

#include "route_dev.cuh"
#include "scaled.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;      // tokens per CTA, a warp each

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

struct Score {
    int kind;
    double top, inv;           // softmax: the largest logit and 1 / sum exp(l - top)
    __device__ __forceinline__ double operator()(float l) const {
        return kind == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)l))
                                         : exp((double)l - top) * inv;
    }
};

// One warp per token; its row of 64-bit values in shared memory.
__global__ void __launch_bounds__(kWarps * 32) k_scored_topk(
    const float *__restrict__ logits, int T, int E, int k, const moe_route_rule rule,
    int32_t *ids, float *w, uint32_t *status) {
    extern __shared__ double s_rows[];
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + wid;
    if (t >= T) return;
    double *row = s_rows + (size_t)wid * E;
    const float *src = logits + (size_t)t * E;
    const float *bias = rule.d_bias;
    ids += (size_t)t * k;
    w += (size_t)t * k;

    bool fin = true;
    float top = -INFINITY;
    for (int e = lane; e < E; e += 32) {
        const float l = src[e];
        fin = fin && isfinite(l) && (!bias || isfinite(bias[e]));
        top = fmaxf(top, l);
    }
    if (!__all_sync(kFull, fin)) {
        if (lane < k) {
            ids[lane] = lane;
            w[lane] = __fdiv_rn(1.0f, (float)k);
        }
        if (lane == 0) set_status(status, MOE_ERR_NONFINITE);
        return;
    }
    Score score{rule.score, 0.0, 1.0};
    if (rule.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        double sum = 0.0;
        for (int e = lane; e < E; e += 32) sum += exp((double)src[e] - (double)top);
        score.top = top;
        score.inv = 1.0 / warp_sum(sum);
    }
    // the order's values: v with a bias, else the logits
    for (int e = lane; e < E; e += 32)
        row[e] = bias ? score(src[e]) + (double)bias[e] : (double)src[e];
    __syncwarp();
    if (rule.n_group > 1) {
        const int per = E / rule.n_group;
        double mine = -INFINITY;             // lane g: the value of group g
        for (int g = 0; g < rule.n_group; g++) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int i = lane; i < per; i += 32) {
                const double v = row[g * per + i];
                b2 = fmax(b2, fmin(b1, v));
                b1 = fmax(b1, v);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const double o1 = __shfl_xor_sync(kFull, b1, o);
                const double o2 = __shfl_xor_sync(kFull, b2, o);
                b2 = fmax(fmin(b1, o1), fmax(b2, o2));
                b1 = fmax(b1, o1);
            }
            // without a bias the row holds logits; one value is ordered as its score is
            if (!bias && rule.group_top == 2) {
                b1 = score((float)b1);
                b2 = score((float)b2);
            }
            if (lane == g) mine = rule.group_top == 2 ? b1 + b2 : b1;
        }
        int rank = 0;
        for (int g = 0; g < rule.n_group; g++) {
            const double o = __shfl_sync(kFull, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        const unsigned keep = __ballot_sync(kFull, lane < rule.n_group && rank < rule.topk_group);
        for (int e = lane; e < E; e += 32)
            if (!((keep >> (e / per)) & 1u)) row[e] = -INFINITY;
        __syncwarp();
    }
    int my_id = 0;
    for (int j = 0; j < k; j++) {
        double bv = -INFINITY;
        int bi = INT_MAX;
        for (int e = lane; e < E; e += 32) {     // ascending e: '>' keeps the lower id
            const double v = row[e];
            if (v > bv) {
                bv = v;
                bi = e;
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const double ov = __shfl_xor_sync(kFull, bv, o);
            const int oi = __shfl_xor_sync(kFull, bi, o);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        if (lane == j) my_id = bi;
        if (lane == (bi & 31)) row[bi] = -INFINITY;   // taken (every other value is larger)
        __syncwarp();
    }
    const double s = lane < k ? score(src[my_id]) : 0.0;
    const double sum = warp_sum(s);
    if (lane < k) {
        const double r = rule.renorm ? (sum > 0.0 ? s / sum : 0.0) : s;
        ids[lane] = my_id;
        w[lane] = (float)(r * (double)rule.scale);
    }
}

}  // namespace

cudaError_t launch_route_scored(const float *logits, int T, int E, int k,
                                const moe_route_rule &rule, int32_t *ids, float *w,
                                int32_t *counts, int32_t *offsets, int32_t *perm,
                                int32_t *inv_perm, uint32_t *status, void *ws, cudaStream_t st) {
    const size_t smem = (size_t)kWarps * E * sizeof(double);
    cudaError_t err = ensure_smem(k_scored_topk, smem);
    if (err != cudaSuccess) return err;
    k_scored_topk<<<(T + kWarps - 1) / kWarps, kWarps * 32, smem, st>>>(logits, T, E, k, rule, ids,
                                                                       w, status);
    note_launches(1);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const RouteWs L = route_ws(T, E, k);
    uint8_t *p = static_cast<uint8_t *>(ws);
    return launch_group(ids, T, k, E, 0, counts, offsets, perm, inv_perm,
                        reinterpret_cast<int32_t *>(p + L.chunk_counts),
                        reinterpret_cast<int32_t *>(p + L.chunk_base),
                        reinterpret_cast<Job *>(p + L.jobs),
                        reinterpret_cast<int32_t *>(p + L.njobs), st);
}

}  // namespace moe
