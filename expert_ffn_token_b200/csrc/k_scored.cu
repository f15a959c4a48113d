// k_scored.cu -- routing by scores: softmax or sigmoid of the logits, a balance bias that takes
// part in the choice alone, groups of experts of which the best stay, top-k, weights from the
// chosen scores; then the grouping of the (token, slot) pairs by expert.
//
// The choice is that of 64-bit scores, so that a near-tie is decided as the formula decides it,
// whatever the order of a sum or the last bits of an fp32 exponential would say.  Only what may
// be chosen pays for 64 bits (k_scored_rows, a warp per token, the row in registers):
//   - the k-th largest of the 32 lanes' own maxima is a bound that the k chosen reach, so the
//     experts at or above it (for fp32 scores: above it less twice the error there) hold the choice;
//     there are seldom more than a dozen;
//   - these candidates, one per lane, get 64-bit scores and are sorted by (value, id);
//   - groups are ranked by fp32 sums, and by 64-bit ones where two lie within the error;
//   - a row with more than 32 candidates (ties, mostly masked rows) takes 64-bit rounds over all.
// Without a bias the order is that of the logits, which needs no scores.
//
// Grouping (the order of a3): counts per chunk of 64 tokens come out of the routing kernel's shared
// memory, a second kernel turns them into places per chunk, a third writes the permutation.  Up to
// one chunk is routed and grouped by one CTA in one launch.
//
// 8192 tokens of 512 experts in 8 groups take 45 us on the device, 38.6 us of it k_scored_rows alone
// (16.8 MB), which is neither bound by the logits' bytes nor by instructions alone: 2418 a token are
// 33,500 issue slots a scheduler of its 75,200 clocks.  The rest is 128 CTAs for 148 SMs, two tokens
// a warp in turn, each a chain of dependent reductions, and at 512 experts spills (64 registers).  One
// token of 256 experts takes 5.0 us.
#include <math.h>

#include "ptx.cuh"
#include "route_dev.cuh"
#include "scaled.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;             // k_scored_wide: tokens per CTA, a warp each
constexpr int kMaxNV = 32;            // experts per lane held in registers (1024 experts)
// k_scored_rows: threads for a chunk of 64 tokens, a warp per token at a time
constexpr int row_threads(int nv) { return nv <= 16 ? 1024 : 512; }

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

// An order-preserving integer of a float (no NaN).
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);        // -0 and 0 are one value
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Rounds of argmax over v[NV] per lane (element i of a lane is expert lane + 32 i), ties to the
// lower id; returns the j-th choice in lane j.
template <int NV, typename V>
__device__ __noinline__ int select_rounds(V (&v)[NV], int k) {
    const int lane = threadIdx.x & 31;
    int mine = 0;
    for (int j = 0; j < k; j++) {
        V bv = -INFINITY;
        int bi = INT_MAX;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (v[i] > bv) {
                bv = v[i];
                bi = lane + 32 * i;
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const V ov = __shfl_xor_sync(kFull, bv, o);
            const int oi = __shfl_xor_sync(kFull, bi, o);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        if (lane == j) mine = bi;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (bi == lane + 32 * i) v[i] = -INFINITY;   // taken (every other value is larger)
    }
    return mine;
}

// The two largest values of a lane's group: values come from get(element).
template <typename V>
struct Best {
    V b1, b2;
    __device__ __forceinline__ V value(int top) const { return top == 2 ? b1 + b2 : b1; }
};
template <typename V, typename Get>
__device__ __forceinline__ Best<V> group_best(int per, int first, int step, int width, Get get) {
    V b1 = -INFINITY, b2 = -INFINITY;
    for (int i = first; i < per; i += step) {
        const V v = get(i);
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
    }
    for (int o = width / 2; o >= 1; o >>= 1) {
        const V o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
        b2 = fmax(fmin(b1, o1), fmax(b2, o2));
        b1 = fmax(b1, o1);
    }
    return {b1, b2};
}

// Which groups stay (a bit each), from lane g's value of group g.
template <typename V>
__device__ __forceinline__ unsigned keep_groups(V mine, int n_group, int topk_group) {
    const int lane = threadIdx.x & 31;
    int rank = 0;
    for (int g = 0; g < n_group; g++) {
        const V o = __shfl_sync(kFull, mine, g);
        rank += o > mine || (o == mine && g < lane);
    }
    return __ballot_sync(kFull, lane < n_group && rank < topk_group);
}

// Whether every kept group's value is above every dropped one's, each up to err off.  A sum past
// fp32 is known to be past its largest value only.
__device__ __forceinline__ bool keep_certain(float mine, float err, unsigned keep, int n_group) {
    constexpr float kMost = 3.402823466e+38f;
    const int lane = threadIdx.x & 31;
    const bool in = lane < n_group, kept = (keep >> lane) & 1u;
    const float m = fminf(fmaxf(mine, -kMost), kMost);
    float lo = in && kept ? m - err : INFINITY, hi = in && !kept ? m + err : -INFINITY;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    }
    return lo > hi;
}

// Bound on what an fp32 value (score plus bias) is off by: a score is at most 1 and a few roundings
// off, the sum rounds once more.  It goes by the value itself, not by the largest bias: one expert
// masked by -1e9 must not blur the others.
__device__ __forceinline__ float value_err(float v) { return 0x1p-19f * (1.0f + fabsf(v)); }

// One token by one warp.  row: E + E / 32 floats of shared memory of the warp's own (groups), cand:
// 32 ints.  ids and w: k entries each (lane j writes entry j).
template <int NV>
__device__ void route_row(const float *__restrict__ src, int E, int k, const moe_route_rule &rule,
                          float *row, int *cand, int32_t *ids, float *w, uint32_t *status) {
    const int lane = threadIdx.x & 31;
    const float *bias = rule.d_bias;
    const bool sigmoid = rule.score == MOE_SCORE_SIGMOID;
    float l[NV], top = -INFINITY;
    uint32_t mag = 0;                     // the largest magnitude: not finite from 0x7f800000 on
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = lane + 32 * i;
        l[i] = -INFINITY;
        if (e < E) {
            l[i] = __ldg(src + e);
            mag = max(mag, __float_as_uint(l[i]) & 0x7fffffffu);
        }
        top = fmaxf(top, l[i]);
    }
    if (bias) {
        uint32_t b = 0;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + 32 * i;
            if (e < E) b = max(b, __float_as_uint(__ldg(bias + e)) & 0x7fffffffu);
        }
        mag = max(mag, b);
    }
    if (__any_sync(kFull, mag >= 0x7f800000u)) {
        if (lane < k) {
            ids[lane] = lane;
            w[lane] = __fdiv_rn(1.0f, (float)k);
        }
        if (lane == 0) set_status(status, MOE_ERR_NONFINITE);
        return;
    }
    Score score{rule.score, 0.0, 1.0};
    float inv32 = 1.0f;
    if (!sigmoid) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        score.top = top;
        if (bias || !rule.renorm) {       // the sum counts in v or in the weights: 64 bits
            double sum = 0.0;
#pragma unroll 1
            for (int e = lane; e < E; e += 32) sum += exp((double)__ldg(src + e) - (double)top);
            score.inv = 1.0 / warp_sum(sum);
        } else if (rule.group_top == 2) { // a common factor of the group sums
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++) sum += expf(l[i] - top);
            score.inv = 1.0 / warp_sum((double)sum);
        }
        inv32 = (float)score.inv;
    }
    // fp32 values: scores plus bias, at most value_err from the 64-bit ones
    const bool grouped = rule.n_group > 1;
    const bool need = bias || (grouped && rule.group_top == 2);
    float v[NV];
    if (need) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + 32 * i;
            const float s = sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l[i]))
                                    : __expf(l[i] - top) * inv32;
            v[i] = e < E ? s + (bias ? __ldg(bias + e) : 0.f) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] = l[i];
    }
    unsigned keep = ~0u;
    int per = E;
    if (grouped) {
        per = E / rule.n_group;
        const bool lined = per % 32 == 0;             // a group is whole registers of the warp
        float value = -INFINITY, err = 0.f;           // lane g: the value of group g, its error
        int width = 32;                               // else: lanes per group
        while (width > 1 && 32 / width < rule.n_group) width >>= 1;
        const int g = lane / width, base = g * per;
        const bool mine = g < rule.n_group;
        if (lined) {
            const int regs = per >> 5;
            int left = regs, at_group = 0;
            uint32_t b1 = 0, b2 = 0;                  // this lane's two largest of the group
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t x = order_key(v[i]);
                b2 = max(b2, min(b1, x));
                b1 = max(b1, x);
                if (--left == 0) {                    // the group's last register
                    const uint32_t m1 = __reduce_max_sync(kFull, b1);
                    Best<float> best{key_value(m1), 0.f};
                    if (rule.group_top == 2) {
                        const unsigned at = __ballot_sync(kFull, b1 == m1);
                        const uint32_t m2 = __reduce_max_sync(kFull, b1 == m1 ? b2 : b1);
                        best.b2 = key_value(at & (at - 1) ? m1 : m2);
                    }
                    if (lane == at_group) {
                        value = best.value(rule.group_top);
                        err = value_err(best.b1) + value_err(best.b2);
                    }
                    at_group++;
                    left = regs;
                    b1 = b2 = 0;
                }
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int e = lane + 32 * i;
                if (e < E) row[e + (e >> 5)] = v[i];
            }
            __syncwarp();
            Best<float> best = group_best<float>(mine ? per : 0, lane % width, width, width,
                                                 [&](int i) {
                                                     const int e = base + i;
                                                     return row[e + (e >> 5)];
                                                 });
            if (rule.group_top == 1) best.b2 = 0.f;
            value = __shfl_sync(kFull, best.value(rule.group_top), (lane * width) & 31);
            err = __shfl_sync(kFull, value_err(best.b1) + value_err(best.b2), (lane * width) & 31);
        }
        keep = keep_groups(value, rule.n_group, rule.topk_group);
        if (need && rule.topk_group < rule.n_group &&
            !keep_certain(value, err, keep, rule.n_group)) {
            const double exact =
                group_best<double>(mine ? per : 0, lane % width, width, width, [&](int i) {
                    const int e = base + i;
                    return score(__ldg(src + e)) + (bias ? (double)__ldg(bias + e) : 0.0);
                }).value(rule.group_top);
            keep = keep_groups(__shfl_sync(kFull, exact, (lane * width) & 31), rule.n_group,
                               rule.topk_group);
        }
    }
    // the order's values; experts of dropped groups and past the end are out
    const uint32_t magic = per > 1 ? (uint32_t)(0xffffffffu / (uint32_t)per + 1u) : 0u;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = lane + 32 * i;
        if (!bias) v[i] = l[i];
        if (grouped) {
            const int g = per > 1 ? (int)__umulhi((uint32_t)e, magic) : e;
            if (!((keep >> (g & 31)) & 1u)) v[i] = -INFINITY;
        }
        best = max(best, order_key(v[i]));
    }
    // the k-th largest lane maximum (or a lower value, where lanes tie)
    uint32_t bound = 0, left = best;
    for (int j = 0; j < k; j++) {
        bound = __reduce_max_sync(kFull, left);
        if (left == bound) left = 0;
    }
    float least = -3.402823466e+38f;      // every finite value: fewer than k lanes hold any
    if (bound > order_key(-INFINITY)) {
        // k experts are at least the bound, less its error; what may reach that is off by as much
        // again (an error grows by 2^-24 of what the value changes by, which the bound covers)
        least = key_value(bound);
        if (bias) least -= 2.0f * value_err(least);
    }
    int held = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) held += v[i] >= least;
    int at = held;                        // places by a prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += x;
    }
    const int n = __shfl_sync(kFull, at, 31);
    at -= held;
    if (n <= 32) {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (v[i] >= least) cand[at++] = lane + 32 * i;
    }
    __syncwarp();
    int my_id = 0;
    double s = 0.0;
    if (n > 32) {
        if (bias) {
            double d[NV];
#pragma unroll 1
            for (int i = 0; i < NV; i++) {
                const int e = lane + 32 * i;
                const double x = e < E ? score(__ldg(src + e)) + (double)__ldg(bias + e) : 0.0;
#pragma unroll
                for (int q = 0; q < NV; q++)
                    if (q == i) d[q] = v[q] > -INFINITY ? x : -INFINITY;
            }
            my_id = select_rounds<NV, double>(d, k);
        } else {
            float c[NV];                   // a copy: the call takes an address
#pragma unroll
            for (int i = 0; i < NV; i++) c[i] = v[i];
            my_id = select_rounds<NV, float>(c, k);
        }
    } else {
        // one candidate per lane, sorted by (value descending, id ascending); the lane a candidate
        // came from rides in the id's low bits
        double d = -INFINITY, own = 0.0;
        int tag = INT_MAX;
        if (lane < n) {
            const int id = cand[lane];
            const float x = __ldg(src + id);
            tag = (id << 5) | lane;
            if (bias || sigmoid) own = score(x);
            d = bias ? own + (double)__ldg(bias + id) : (double)x;
            if (!bias && !sigmoid) own = d;
        }
        const int most = n <= 16 ? 16 : 32;
#pragma unroll
        for (int size2 = 2; size2 <= 32; size2 <<= 1) {
            if (size2 > most) break;
#pragma unroll
            for (int o = size2 >> 1; o >= 1; o >>= 1) {
                const double od = __shfl_xor_sync(kFull, d, o);
                const int oi = __shfl_xor_sync(kFull, tag, o);
                const bool before = od > d || (od == d && oi < tag);     // the other sorts first
                const bool first = ((lane & size2) == 0) == ((lane & o) == 0);
                if (before == first) {
                    d = od;
                    tag = oi;
                }
            }
        }
        my_id = tag >> 5;
        const double s0 = __shfl_sync(kFull, own, tag & 31);
        s = bias || sigmoid ? s0 : exp(s0 - score.top) * score.inv;
    }
    __syncwarp();
    if (n > 32) s = lane < k ? score(__ldg(src + my_id)) : 0.0;
    if (lane >= k) s = 0.0;
    double r = s;
    if (rule.renorm) {
        const double sum = warp_sum(s);
        r = sum > 0.0 ? s / sum : 0.0;
    }
    if (lane < k) {
        ids[lane] = my_id;
        w[lane] = (float)(r * (double)rule.scale);
    }
}

struct RouteOut {
    int32_t *ids;
    float *w;
    int32_t *counts, *offsets, *perm, *inv_perm;
    uint32_t *status;
};

// Places of a chunk's pairs, in ascending (token, slot): base[e] is the next place of expert e.
// One warp.
__device__ __forceinline__ void place_pairs(const int *pairs, int n, int first, int *base,
                                            int32_t *perm, int32_t *inv_perm) {
    const int lane = threadIdx.x & 31;
    for (int a0 = 0; a0 < n; a0 += 32) {
        const int a = a0 + lane;
        const bool act = a < n;
        const int e = act ? pairs[a] : -1;
        const unsigned peers = __match_any_sync(kFull, e);
        const int leader = __ffs(peers) - 1;
        if (act) {
            const int pos = base[e] + __popc(peers & ((1u << lane) - 1u));
            perm[pos] = first + a;
            if (inv_perm) inv_perm[first + a] = pos;
        }
        __syncwarp();
        if (act && lane == leader) base[e] += __popc(peers);
        __syncwarp();
    }
}

// grid: chunks of 64 tokens.  One chunk in all (kWhole): also the grouping.
template <int NV, bool kWhole>
__global__ void __launch_bounds__(row_threads(NV), 1)
    k_scored_rows(const float *__restrict__ logits, int T, int E, int k, const moe_route_rule rule,
                  const RouteOut o, int32_t *chunk_counts) {
    constexpr int kThreads = row_threads(NV), kTokens = kThreads / 32;
    ptx::launch_dependents();
    extern __shared__ float s_rows[];            // [warps][E + E / 32], when there are groups
    __shared__ int s_cnt[NV * 32];
    __shared__ int s_ids[kChunk * kMaxK];
    __shared__ int s_cand[kTokens][32];
    __shared__ int s_warp[33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * kChunk, nt = min(kChunk, T - t0);
    for (int e = threadIdx.x; e < E; e += kThreads) s_cnt[e] = 0;
    for (int t = warp; t < nt; t += kTokens) {
        int32_t *ids = s_ids + t * k;
        route_row<NV>(logits + (size_t)(t0 + t) * E, E, k, rule,
                      s_rows + (size_t)warp * (E + (E + 31) / 32), s_cand[warp], ids,
                      o.w + (size_t)(t0 + t) * k, o.status);
        __syncwarp();
        if (lane < k) o.ids[(size_t)(t0 + t) * k + lane] = ids[lane];
    }
    __syncthreads();
    for (int a = threadIdx.x; a < nt * k; a += kThreads) atomicAdd(&s_cnt[s_ids[a]], 1);
    __syncthreads();
    if constexpr (kWhole) {
        for (int e = threadIdx.x; e < E; e += kThreads) o.counts[e] = s_cnt[e];
        const int total = block_exclusive_scan<kThreads>(s_cnt, E, s_warp);
        for (int e = threadIdx.x; e < E; e += kThreads) o.offsets[e] = s_cnt[e];
        if (threadIdx.x == 0) o.offsets[E] = total;
        __syncthreads();
        if (warp == 0) place_pairs(s_ids, nt * k, 0, s_cnt, o.perm, o.inv_perm);
    } else {
        for (int e = threadIdx.x; e < E; e += kThreads)
            chunk_counts[(size_t)blockIdx.x * E + e] = s_cnt[e];
    }
}

// grid: 32 experts a CTA; thread (segment, expert).  Totals, and per chunk how many pairs of the
// expert earlier chunks hold.
__global__ void __launch_bounds__(1024)
    k_scored_chunks(const int32_t *__restrict__ chunk_counts, int n_chunks, int E,
                    int32_t *chunk_base, int32_t *counts) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    __shared__ int s_sum[32][33];
    const int seg = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
    const int per = (n_chunks + 31) / 32, c0 = seg * per, c1 = min(n_chunks, c0 + per);
    int sum = 0;
    if (e < E) {
#pragma unroll 4
        for (int c = c0; c < c1; c++) sum += __ldcg(chunk_counts + (size_t)c * E + e);
    }
    s_sum[seg][lane] = sum;
    __syncthreads();
    int run = 0, all = 0;
#pragma unroll
    for (int s = 0; s < 32; s++) {
        const int x = s_sum[s][lane];
        run += s < seg ? x : 0;
        all += x;
    }
    if (e >= E) return;
    if (seg == 0) counts[e] = all;
    for (int c = c0; c < c1; c++) {
        chunk_base[(size_t)c * E + e] = run;
        run += __ldcg(chunk_counts + (size_t)c * E + e);
    }
}

// grid: chunks.  Every CTA adds up the experts' totals (the first writes the offsets) and places
// its chunk's pairs.
__global__ void __launch_bounds__(256)
    k_scored_place(int T, int E, int k, const int32_t *__restrict__ chunk_base, const RouteOut o) {
    extern __shared__ int s_base[];              // [E]
    __shared__ int s_ids[kChunk * kMaxK];
    __shared__ int s_warp[33];
    const int t0 = blockIdx.x * kChunk, n = min(kChunk, T - t0) * k;
    // the ids were complete before k_scored_chunks let this kernel start
    for (int a = threadIdx.x; a < n; a += 256) s_ids[a] = __ldcg(o.ids + (size_t)t0 * k + a);
    ptx::grid_dependency_wait();
    for (int e = threadIdx.x; e < E; e += 256) s_base[e] = __ldcg(o.counts + e);
    __syncthreads();
    const int total = block_exclusive_scan<256>(s_base, E, s_warp);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += 256) o.offsets[e] = s_base[e];
        if (threadIdx.x == 0) o.offsets[E] = total;
        __syncthreads();
    }
    for (int e = threadIdx.x; e < E; e += 256)
        s_base[e] += __ldcg(chunk_base + (size_t)blockIdx.x * E + e);
    __syncthreads();
    if (threadIdx.x < 32) place_pairs(s_ids, n, t0 * k, s_base, o.perm, o.inv_perm);
}

// More experts than registers hold: one warp per token, its row of 64-bit values in shared memory.
__global__ void __launch_bounds__(kWarps * 32)
    k_scored_wide(const float *__restrict__ logits, int T, int E, int k, const moe_route_rule rule,
                  int32_t *ids, float *w, uint32_t *status) {
    extern __shared__ double s_wide[];
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + wid;
    if (t >= T) return;
    double *row = s_wide + (size_t)wid * E;
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
            Best<double> best = group_best<double>(per, lane, 32, 32,
                                                   [&](int i) { return row[g * per + i]; });
            // without a bias the row holds logits; one value is ordered as its score is
            if (!bias && rule.group_top == 2)
                best = {score((float)best.b1), score((float)best.b2)};
            if (lane == g) mine = best.value(rule.group_top);
        }
        const unsigned keep = keep_groups(mine, rule.n_group, rule.topk_group);
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

template <int NV>
cudaError_t run_rows(const float *logits, int T, int E, int k, const moe_route_rule &rule,
                     const RouteOut &o, int32_t *chunk_counts, cudaStream_t st) {
    const size_t smem = rule.n_group > 1 ? (size_t)(row_threads(NV) / 32) * (E + (E + 31) / 32) * sizeof(float) : 0;
    const int n_chunks = (T + kChunk - 1) / kChunk;
    auto kernel = n_chunks == 1 ? k_scored_rows<NV, true> : k_scored_rows<NV, false>;
    cudaError_t err = ensure_smem(kernel, smem);
    if (err != cudaSuccess) return err;
    kernel<<<n_chunks, row_threads(NV), smem, st>>>(logits, T, E, k, rule, o, chunk_counts);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_scored(const float *logits, int T, int E, int k,
                                const moe_route_rule &rule, int32_t *ids, float *w,
                                int32_t *counts, int32_t *offsets, int32_t *perm,
                                int32_t *inv_perm, uint32_t *status, void *ws, cudaStream_t st) {
    const RouteWs L = route_ws(T, E, k);
    uint8_t *p = static_cast<uint8_t *>(ws);
    int32_t *chunk_counts = reinterpret_cast<int32_t *>(p + L.chunk_counts);
    int32_t *chunk_base = reinterpret_cast<int32_t *>(p + L.chunk_base);
    if (E > 32 * kMaxNV) {
        const size_t smem = (size_t)kWarps * E * sizeof(double);
        cudaError_t err = ensure_smem(k_scored_wide, smem);
        if (err != cudaSuccess) return err;
        k_scored_wide<<<(T + kWarps - 1) / kWarps, kWarps * 32, smem, st>>>(logits, T, E, k, rule,
                                                                           ids, w, status);
        note_launches(1);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        return launch_group(ids, T, k, E, 0, counts, offsets, perm, inv_perm, chunk_counts,
                            chunk_base, reinterpret_cast<Job *>(p + L.jobs),
                            reinterpret_cast<int32_t *>(p + L.njobs), st);
    }
    const RouteOut o{ids, w, counts, offsets, perm, inv_perm, status};
    cudaError_t err;
    if (E <= 128)
        err = run_rows<4>(logits, T, E, k, rule, o, chunk_counts, st);
    else if (E <= 256)
        err = run_rows<8>(logits, T, E, k, rule, o, chunk_counts, st);
    else if (E <= 512)
        err = run_rows<16>(logits, T, E, k, rule, o, chunk_counts, st);
    else
        err = run_rows<kMaxNV>(logits, T, E, k, rule, o, chunk_counts, st);
    if (err != cudaSuccess) return err;
    const int n_chunks = (T + kChunk - 1) / kChunk;
    if (n_chunks == 1) return cudaSuccess;
    err = launch_behind(k_scored_chunks, dim3((E + 31) / 32), 1024, 0, st, chunk_counts, n_chunks, E,
                        chunk_base, counts);
    if (err != cudaSuccess) return err;
    return launch_behind(k_scored_place, dim3(n_chunks), 256, (size_t)E * sizeof(int), st, T, E, k,
                         chunk_base, o);
}

}  // namespace moe
