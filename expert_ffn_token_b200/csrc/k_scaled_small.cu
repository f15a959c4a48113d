// k_scaled_small.cu -- products of scaled (e4m3, 128-block) operands for few tokens, where the
// weights are read once and their bytes set the time.
//
// out[m][n] = sum_b as[b][m] bs[n/128][b] * (sum over the block's 128 k of a[m][k] w[n][k]).
// The inner sums run on mma.sync.m16n8k32 (e4m3 operands, fp32 accumulator): a warp holds 16
// weight rows against 8 token columns, and a block's sum is scaled and added up in fp32.  A sum
// over k does not depend on the order of k, so the operands are loaded in an order that suits
// the loads: lane (g, c) reads 16 contiguous bytes of rows g and g + 8 at byte 16 c of each
// 64-byte half block, straight into the fragments of two MMAs, and the activations are permuted
// likewise.  No shared memory, no conversion of weights.
//
// Where there are few rows to read, the weights of 16 rows are split over k among a CTA's 8 warps,
// whose partial sums meet in shared memory in the order of the warps, so results repeat.
//
// The experts' layer, one token (two kernels): k_one_gateup splits 16 gate and 16 up rows of one
// routed expert over k, every warp quantising the blocks of x that it needs; k_one_down gives 16
// output rows of all the token's experts to one CTA, which combines them, and starts its weight
// loads before the first kernel has ended.
// 2 to 4 tokens (three kernels): k_few_prep lists the distinct experts with the tokens routed to
// them and quantises x once; k_few_gateup takes 128 ffn values of one expert per CTA, 16 rows and
// all of k per warp, so that h can be quantised in place; k_few_down takes 16 output rows over all
// experts.  An expert's rows are read once for all its tokens, which are the MMA's columns.
//
// On the device: one row times 1280 x 2560 2.8 us (3.3 MB: a launch and one trip to memory); one
// token of 8 experts, hidden 2048, ffn 512, 8.7 us (25 MB, 2.9 TB/s); 3 tokens of 10 of 512 experts
// and the shared one, hidden 2560, ffn 640, 47 us (124 MB): list 5, gate/up 22.5, down 19 us, a third
// of the issue slots and 2.6 TB/s: few CTAs, and the down kernel spills 156 bytes a thread.
#include <algorithm>

#include "ptx.cuh"
#include "scaled.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;                 // weight rows per CTA

// One 64-byte half block: rows g (lo) and g + 8 (hi), columns' 16 bytes x.
__device__ __forceinline__ void mma64(float (&c)[4], const uint4 &lo, const uint4 &hi,
                                      const uint4 &x) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(lo.x), "r"(hi.x), "r"(lo.y), "r"(hi.y), "r"(x.x), "r"(x.y));
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(lo.z), "r"(hi.z), "r"(lo.w), "r"(hi.w), "r"(x.z), "r"(x.w));
}

// 16 bytes at p, or zeros: one predicated load, so that a run of them issues without a branch or a
// use in between (with the bytes masked as they came, a block's eight loads took 4 us).
__device__ __forceinline__ uint4 ldg16_if(const uint8_t *p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)in));
    return v;
}

// Keep the first n (0..16) bytes of v.
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
    uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int m = n - 4 * i;
        r[i] = m >= 4 ? r[i] : m <= 0 ? 0u : r[i] & ((1u << (8 * m)) - 1u);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// One block's 16 bytes per half of a row (at column k and k + 64 of K columns; zeros past the end,
// where K is a multiple of 16 or the bytes are cut afterwards: the row's stride is a multiple of
// 16, so a chunk that starts inside it lies inside it).
struct Half2 {
    uint4 a, b;
    __device__ __forceinline__ void load(const uint8_t *p, bool row, int k, int K) {
        a = ldg16_if(p + k, row && k < K);
        b = ldg16_if(p + k + 64, row && k + 64 < K);
    }
    __device__ __forceinline__ void cut(int k, int K) {
        a = keep_bytes(a, K - k);
        b = keep_bytes(b, K - k - 64);
    }
};

// The partial sums red[warp][col * 16 + row] of entry i, added in warp order.
__device__ __forceinline__ float sum_warps(const float (*red)[kTile * 8], int i) {
    float s = red[0][i];
#pragma unroll
    for (int w = 1; w < kWarps; w++) s += red[w][i];
    return s;
}

__device__ __forceinline__ void put_frag(float *red, const float (&c)[4], int g, int tig) {
    red[(2 * tig) * kTile + g] = c[0];
    red[(2 * tig + 1) * kTile + g] = c[1];
    red[(2 * tig) * kTile + g + 8] = c[2];
    red[(2 * tig + 1) * kTile + g + 8] = c[3];
}

// ------------------------------------------------------------------ one matrix

// grid (rows of weights / 16): up to 8 rows of a, the MMA's columns.
static_assert(kSmallT == 8, "a row of a per MMA column");
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_scaled_rows(const ScaledMatmulArgs a) {
    __shared__ float red[kWarps][kTile * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int n0 = blockIdx.x * kTile;
    const int nb = sblocks(a.K);
    const uint8_t *lo = a.b + (int64_t)min(n0 + g, a.N - 1) * a.ldb;
    const uint8_t *hi = a.b + (int64_t)min(n0 + g + 8, a.N - 1) * a.ldb;
    const uint8_t *xr = a.a + (int64_t)min(g, a.M - 1) * a.lda;
    const float *ws = a.bs + (int64_t)(n0 / kSBlk) * nb;
    const int c0 = 2 * tig, c1 = c0 + 1;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    struct Block {
        Half2 l, h, x;
        float sw, s0, s1;
    } q[2];
    auto load = [&](Block &k, int b) {
        const int k0 = b * kSBlk + 16 * tig;
        const bool in = b < nb;
        k.l.load(lo, in && n0 + g < a.N, k0, a.K);
        k.h.load(hi, in && n0 + g + 8 < a.N, k0, a.K);
        k.x.load(xr, in && g < a.M, k0, a.K);
        k.sw = in ? __ldg(ws + b) : 0.f;
        k.s0 = in && c0 < a.M ? __ldg(a.as + b * a.ldas + c0) : 0.f;
        k.s1 = in && c1 < a.M ? __ldg(a.as + b * a.ldas + c1) : 0.f;
    };
    auto add = [&](Block &k, int b) {
        if (b >= nb) return;
        const int k0 = b * kSBlk + 16 * tig;
        if ((b + 1) * kSBlk > a.K) {
            k.l.cut(k0, a.K);
            k.h.cut(k0, a.K);
            k.x.cut(k0, a.K);
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma64(c, k.l.a, k.h.a, k.x.a);
        mma64(c, k.l.b, k.h.b, k.x.b);
        const float s0 = k.s0 * k.sw, s1 = k.s1 * k.sw;
        acc[0] = fmaf(c[0], s0, acc[0]);
        acc[1] = fmaf(c[1], s1, acc[1]);
        acc[2] = fmaf(c[2], s0, acc[2]);
        acc[3] = fmaf(c[3], s1, acc[3]);
    };
    load(q[0], warp);
    for (int b = warp; b < nb; b += 2 * kWarps) {
        load(q[1], b + kWarps);
        add(q[0], b);
        load(q[0], b + 2 * kWarps);
        add(q[1], b + kWarps);
    }
    put_frag(red[warp], acc, g, tig);
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kTile * 8) {
        const int m = i / kTile, n = n0 + i % kTile;
        if (m < a.M && n < a.N)
            static_cast<T *>(a.out)[m * a.ldo + n] = from_f32<T>(sum_warps(red, i));
    }
}

// ------------------------------------------------------------------ the experts, one token

// Weight rows g and g + 8 of one block of k.
struct Rows16 {
    Half2 lo, hi;
    __device__ __forceinline__ void load(const uint8_t *p, int64_t pitch, bool in, int k, int K) {
        lo.load(p, in, k, K);
        hi.load(p + 8 * pitch, in, k, K);
    }
    __device__ __forceinline__ void multiply(float (&c)[4], const uint4 &x0, const uint4 &x1) const {
        mma64(c, lo.a, hi.a, x0);
        mma64(c, lo.b, hi.b, x1);
    }
};

__device__ __forceinline__ uint32_t byte_word(uint32_t v, int src) {
    return __shfl_sync(0xffffffffu, v, src);
}
// The activation fragment of one token from the packed bytes that quant_block left in the lanes
// (lane l: bytes 4 l .. 4 l + 3): column 0 is the token, the others are zero.
__device__ __forceinline__ void one_column(uint32_t p, uint4 &x0, uint4 &x1) {
    const int lane = threadIdx.x & 31, s = 4 * (lane & 3);
    const uint4 a = make_uint4(byte_word(p, s), byte_word(p, s + 1), byte_word(p, s + 2),
                               byte_word(p, s + 3));
    const uint4 b = make_uint4(byte_word(p, 16 + s), byte_word(p, 17 + s), byte_word(p, 18 + s),
                               byte_word(p, 19 + s));
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    x0 = lane < 4 ? a : zero;
    x1 = lane < 4 ? b : zero;
}

// Slot j's expert: the token's j-th id, the shared expert behind them; -1 (reported) out of range.
__device__ __forceinline__ int one_expert(const ScaledExpertsArgs &a, int j) {
    if (j == a.k) return a.w.n_experts;
    const int e = __ldg(a.ids + j);
    if (e >= 0 && e < a.w.n_experts) return e;
    set_status(a.status, MOE_ERR_BOUNDS);
    return -1;
}

// grid (ffn / 16, slots): h of 16 rows of one slot's expert.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_one_gateup(const ScaledExpertsArgs a) {
    __shared__ float red[2][kWarps][kTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    ptx::launch_dependents();
    const int j = blockIdx.y, e = one_expert(a, j);
    if (e < 0) return;
    const int H = a.w.hidden, F = a.w.ffn, hb = sblocks(H);
    const int f0 = blockIdx.x * kTile;
    const int64_t r0 = (int64_t)e * F + f0 + g;
    const uint8_t *gp = a.w.d_gate + r0 * H, *up = a.w.d_up + r0 * H;
    const int64_t sb = ((int64_t)e * sblocks(F) + f0 / kSBlk) * hb;
    const float *gs = a.w.d_gate_s + sb, *us = a.w.d_up_s + sb;
    float ag[2] = {0.f, 0.f}, au[2] = {0.f, 0.f};      // rows g and g + 8
    for (int b = warp; b < hb; b += kWarps) {
        Rows16 wg, wu;
        wg.load(gp, H, true, b * kSBlk + 16 * tig, H);
        wu.load(up, H, true, b * kSBlk + 16 * tig, H);
        const float sg = __ldg(gs + b), su = __ldg(us + b);
        const int c = b * kSBlk + 4 * lane;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < H) v = load4(static_cast<const T *>(a.x) + c);
        float s;
        bool fin;
        const uint32_t p = quant_block(v, &s, &fin);
        if (!fin && lane == 0) set_status(a.status, MOE_ERR_NONFINITE);
        uint4 x0, x1;
        one_column(p, x0, x1);
        float cg[4] = {0.f, 0.f, 0.f, 0.f}, cu[4] = {0.f, 0.f, 0.f, 0.f};
        wg.multiply(cg, x0, x1);
        wu.multiply(cu, x0, x1);
        ag[0] = fmaf(cg[0], s * sg, ag[0]);
        ag[1] = fmaf(cg[2], s * sg, ag[1]);
        au[0] = fmaf(cu[0], s * su, au[0]);
        au[1] = fmaf(cu[2], s * su, au[1]);
    }
    if (tig == 0) {                                     // column 0 of the fragments
        red[0][warp][g] = ag[0];
        red[0][warp][g + 8] = ag[1];
        red[1][warp][g] = au[0];
        red[1][warp][g + 8] = au[1];
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
        float gv = 0.f, uv = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            gv += red[0][w][threadIdx.x];
            uv += red[1][w][threadIdx.x];
        }
        a.h[(int64_t)j * F + f0 + threadIdx.x] = swiglu(gv, uv);
    }
}

// grid (hidden / 16): 16 output rows over every slot's expert.  Items (slot, block of ffn) go round
// the warps, four at a time.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_one_down(const ScaledExpertsArgs a) {
    constexpr int kBatch = 4;
    __shared__ float red[kWarps][kTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int H = a.w.hidden, F = a.w.ffn, fb = sblocks(F);
    const int n0 = blockIdx.x * kTile;
    const int items = (a.k + a.w.shared) * fb;
    Rows16 w[kBatch];
    float c[kBatch];                       // weight scale times routing weight
    int slot[kBatch];
    auto load = [&](int first) {
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            const int i = first + u * kWarps;
            const int j = min(i, items - 1) / fb, b = min(i, items - 1) - j * fb;
            const int e = i < items ? one_expert(a, j) : -1;
            slot[u] = e >= 0 ? j : -1;
            const int64_t x = max(e, 0);
            w[u].load(a.w.d_down + (x * H + n0 + g) * F, F, e >= 0, b * kSBlk + 16 * tig, F);
            const float r = j < a.k ? __ldg(a.rw + j) : a.gate ? __ldg(a.gate) : 1.0f;
            c[u] = __ldg(a.w.d_down_s + (x * sblocks(H) + n0 / kSBlk) * fb + b) * r;
        }
    };
    load(warp);
    ptx::grid_dependency_wait();           // h is complete
    float acc[2] = {0.f, 0.f};
    for (int first = warp; first < items; first += kBatch * kWarps) {
        if (first != warp) load(first);
        float4 h[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            const int i = first + u * kWarps, col = (i % fb) * kSBlk + 4 * lane;
            h[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot[u] >= 0 && col < F)
                h[u] = __ldcg(reinterpret_cast<const float4 *>(a.h + (int64_t)slot[u] * F + col));
        }
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            if (slot[u] < 0) continue;
            float s;
            bool fin;
            const uint32_t p = quant_block(h[u], &s, &fin);
            if (!fin && lane == 0) set_status(a.status, MOE_ERR_NONFINITE);
            uint4 x0, x1;
            one_column(p, x0, x1);
            float cc[4] = {0.f, 0.f, 0.f, 0.f};
            w[u].multiply(cc, x0, x1);
            acc[0] = fmaf(cc[0], s * c[u], acc[0]);
            acc[1] = fmaf(cc[2], s * c[u], acc[1]);
        }
    }
    if (tig == 0) {
        red[warp][g] = acc[0];
        red[warp][g + 8] = acc[1];
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; q++) s += red[q][threadIdx.x];
        static_cast<T *>(a.out)[n0 + threadIdx.x] = from_f32<T>(s);
    }
}

// ------------------------------------------------------------------ the experts, 2 to 4 tokens

// What k_few_prep leaves in the workspace.
struct FewWs {
    uint8_t *xq;         // [8][hidden]
    float *xs;           // [blocks][8]
    int32_t *njobs;
    int32_t *expert;     // [jobs]: the distinct experts, the shared one last
    int32_t *mask;       // [jobs]: a bit per token routed there
    float *weight;       // [jobs][8]: the weight of the expert's output per token
    uint8_t *hq;         // [jobs][8][ffn]
    float *hs;           // [jobs][8][blocks of ffn]
};

size_t few_layout(int T, int k, int shared, int H, int F, uint8_t *base, FewWs *out) {
    const size_t jobs = (size_t)T * k + (shared ? 1 : 0);
    size_t p = 0;
    auto take = [&](size_t bytes) {
        uint8_t *r = base + p;
        p = (p + bytes + 255) & ~size_t(255);
        return r;
    };
    FewWs w{};
    w.xq = take((size_t)kSmallT * H);
    w.xs = reinterpret_cast<float *>(take((size_t)sblocks(H) * kSmallT * 4));
    w.njobs = reinterpret_cast<int32_t *>(take(4));
    w.expert = reinterpret_cast<int32_t *>(take(jobs * 4));
    w.mask = reinterpret_cast<int32_t *>(take(jobs * 4));
    w.weight = reinterpret_cast<float *>(take(jobs * kSmallT * 4));
    w.hq = take(jobs * kSmallT * F);
    w.hs = reinterpret_cast<float *>(take(jobs * kSmallT * sblocks(F) * 4));
    if (out) *out = w;
    return p;
}

// CTA 0 lists the jobs; the others quantise a block of a token per warp.
template <typename T>
__global__ void __launch_bounds__(256) k_few_prep(const ScaledExpertsArgs a, const FewWs f) {
    ptx::launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x > 0) {
        const int H = a.w.hidden, hb = sblocks(H);
        const int unit = ((int)blockIdx.x - 1) * 8 + warp;
        const int t = unit / hb, b = unit - t * hb;
        if (t >= a.T) return;
        const int c = b * kSBlk + 4 * lane;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < H) v = load4(static_cast<const T *>(a.x) + (int64_t)t * H + c);
        float s;
        bool fin;
        const uint32_t p = quant_block(v, &s, &fin);
        if (c < H) *reinterpret_cast<uint32_t *>(f.xq + (int64_t)t * H + c) = p;
        if (lane == 0) {
            f.xs[b * kSmallT + t] = s;
            if (!fin) set_status(a.status, MOE_ERR_NONFINITE);
        }
        return;
    }
    // the distinct experts in order of first appearance; a thread per (token, slot) pair
    __shared__ int s_ids[kSmallT * kMaxK];
    __shared__ float s_w[kSmallT * kMaxK];
    __shared__ int s_count[8];
    const int A = a.T * a.k, i = threadIdx.x;
    int e = -1;
    if (i < A) {
        e = __ldg(a.ids + i);
        s_w[i] = __ldg(a.rw + i);
        if (e < 0 || e >= a.w.n_experts) {
            e = -1;
            set_status(a.status, MOE_ERR_BOUNDS);
        }
        s_ids[i] = e;
    }
    __syncthreads();
    bool first = e >= 0;
    for (int b = 0; b < i && first; b++) first = s_ids[b] != e;
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_count[warp] = __popc(m);
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 8; w++) {
        base += w < warp ? s_count[w] : 0;
        total += s_count[w];
    }
    if (first) {
        const int j = base + __popc(m & ((1u << lane) - 1u));
        unsigned mask = 0;
        for (int t = 0; t < a.T; t++) {
            float w = 0.f;                 // a token that names the expert twice adds both weights
            for (int q = 0; q < a.k; q++) {
                if (s_ids[t * a.k + q] != e) continue;
                mask |= 1u << t;
                w += s_w[t * a.k + q];
            }
            f.weight[j * kSmallT + t] = w;
        }
        f.expert[j] = e;
        f.mask[j] = (int)mask;
    }
    if (i == 0) {
        *f.njobs = total + a.w.shared;
        if (a.w.shared) {
            f.expert[total] = a.w.n_experts;
            f.mask[total] = (1 << a.T) - 1;
            for (int t = 0; t < a.T; t++)
                f.weight[total * kSmallT + t] = a.gate ? __ldg(a.gate + t) : 1.0f;
        }
    }
}

// 16 bytes that a kernel before this one wrote, or zeros.
__device__ __forceinline__ uint4 ldcg16_if(const uint8_t *p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)in)
        : "memory");
    return v;
}

// grid (blocks of ffn, most jobs): 128 ffn values of one expert, two warps per 16 of them that take
// alternate blocks of k; h quantised.
constexpr int kFewThreads = 512;
__global__ void __launch_bounds__(kFewThreads, 1)
    k_few_gateup(const ScaledExpertsArgs a, const FewWs f) {
    __shared__ float s_part[kWarps][32][8];
    __shared__ uint32_t s_max[kWarps][8];
    const int warp = (threadIdx.x >> 5) & 7, half = threadIdx.x >> 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int j = blockIdx.y;
    if (j >= __ldcg(f.njobs)) return;
    const int e = __ldcg(f.expert + j);
    const unsigned mask = (unsigned)__ldcg(f.mask + j);
    const int H = a.w.hidden, F = a.w.ffn, hb = sblocks(H), fb = sblocks(F);
    const int f0 = blockIdx.x * kSBlk + warp * kTile;
    float ag[4] = {0.f, 0.f, 0.f, 0.f}, au[4] = {0.f, 0.f, 0.f, 0.f};
    if (f0 < F) {
        const int64_t r0 = (int64_t)e * F + f0 + g;
        const uint8_t *gp = a.w.d_gate + r0 * H, *up = a.w.d_up + r0 * H;
        const int64_t sb = ((int64_t)e * fb + blockIdx.x) * hb;
        const float *gs = a.w.d_gate_s + sb, *us = a.w.d_up_s + sb;
        const uint8_t *xr = f.xq + (int64_t)g * H;
        const bool col = g < a.T;
        // everything a block needs is loaded a block ahead, the activations first: a wait for
        // them must not wait for weights that come from HBM after them
        struct Block {
            uint4 x0, x1;
            float2 xs;
            float sg, su;
            Rows16 wg, wu;
        } q[2];
        auto load = [&](Block &k, int b) {
            const int k0 = b * kSBlk + 16 * tig;
            const bool in = b < hb;
            k.x0 = ldcg16_if(xr + k0, in && col && k0 < H);
            k.x1 = ldcg16_if(xr + k0 + 64, in && col && k0 + 64 < H);
            const int bb = min(b, hb - 1);
            k.xs = __ldcg(reinterpret_cast<const float2 *>(f.xs + bb * kSmallT + 2 * tig));
            k.sg = __ldg(gs + bb);
            k.su = __ldg(us + bb);
            k.wg.load(gp, H, in, k0, H);
            k.wu.load(up, H, in, k0, H);
        };
        auto add = [&](const Block &k) {
            float cg[4] = {0.f, 0.f, 0.f, 0.f}, cu[4] = {0.f, 0.f, 0.f, 0.f};
            k.wg.multiply(cg, k.x0, k.x1);
            k.wu.multiply(cu, k.x0, k.x1);
            const float g0 = k.xs.x * k.sg, g1 = k.xs.y * k.sg;
            const float u0 = k.xs.x * k.su, u1 = k.xs.y * k.su;
            ag[0] = fmaf(cg[0], g0, ag[0]);
            ag[1] = fmaf(cg[1], g1, ag[1]);
            ag[2] = fmaf(cg[2], g0, ag[2]);
            ag[3] = fmaf(cg[3], g1, ag[3]);
            au[0] = fmaf(cu[0], u0, au[0]);
            au[1] = fmaf(cu[1], u1, au[1]);
            au[2] = fmaf(cu[2], u0, au[2]);
            au[3] = fmaf(cu[3], u1, au[3]);
        };
        load(q[0], half);
        for (int b = half; b < hb; b += 4) {
            load(q[1], b + 2);
            add(q[0]);
            if (b + 2 >= hb) break;
            load(q[0], b + 4);
            add(q[1]);
        }
    }
    if (half == 1) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            s_part[warp][lane][i] = ag[i];
            s_part[warp][lane][4 + i] = au[i];
        }
    }
    __syncthreads();
    float hv[4] = {0.f, 0.f, 0.f, 0.f};    // rows g, g + 8 by columns 2 tig, 2 tig + 1
    if (half == 0) {
        if (f0 < F) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float gv = ag[i] + s_part[warp][lane][i], uv = au[i] + s_part[warp][lane][4 + i];
                // a column that is not routed here holds another token's products or nothing
                const bool on = (mask >> (2 * tig + (i & 1))) & 1u;
                hv[i] = on ? swiglu(gv, uv) : 0.f;
            }
        }
        // the largest |h| of each column over the CTA's 128 rows
        uint32_t m0 = max(__float_as_uint(hv[0]) & 0x7fffffffu, __float_as_uint(hv[2]) & 0x7fffffffu);
        uint32_t m1 = max(__float_as_uint(hv[1]) & 0x7fffffffu, __float_as_uint(hv[3]) & 0x7fffffffu);
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
            m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        if (g == 0) {
            s_max[warp][2 * tig] = m0;
            s_max[warp][2 * tig + 1] = m1;
        }
    }
    __syncthreads();
    if (half == 1) return;
#pragma unroll
    for (int c = 0; c < 2; c++) {
        const int t = 2 * tig + c;
        uint32_t mx = 0u;
#pragma unroll
        for (int w = 0; w < kWarps; w++) mx = max(mx, s_max[w][t]);
        if (!((mask >> t) & 1u)) continue;
        const bool fin = mx < 0x7f800000u;
        const float sc = fin ? __fdiv_rn(__uint_as_float(mx), kE4M3Max) : 0.f;
        const int64_t row = (int64_t)j * kSmallT + t;
        if (warp == 0 && g == 0) {
            f.hs[row * fb + blockIdx.x] = sc;
            if (!fin) set_status(a.status, MOE_ERR_NONFINITE);
        }
        if (f0 < F) {
            const float4 v = make_float4(hv[c], hv[c + 2], 0.f, 0.f);
            const uint32_t p = sc > 0.f ? quant4(v, sc, __frcp_rn(sc)) : 0u;
            f.hq[row * F + f0 + g] = (uint8_t)p;
            f.hq[row * F + f0 + g + 8] = (uint8_t)(p >> 8);
        }
    }
}

// grid (hidden / 16): 16 output rows for all tokens, over every job.  Items (job, block of ffn) go
// round the warps, two at a time; the first two's weights are loaded before h is complete.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 2)
    k_few_down(const ScaledExpertsArgs a, const FewWs f) {
    constexpr int kBatch = 2;
    __shared__ float red[kWarps][kTile * 8];
    __shared__ int s_expert[kSmallT * kMaxK + 1], s_mask[kSmallT * kMaxK + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int H = a.w.hidden, F = a.w.ffn, fb = sblocks(F);
    const int n0 = blockIdx.x * kTile;
    // the job list was complete before k_few_gateup let this kernel start
    const int njobs = __ldcg(f.njobs), items = njobs * fb;
    for (int j = threadIdx.x; j < max(njobs, 1); j += blockDim.x) {
        s_expert[j] = njobs ? __ldcg(f.expert + j) : 0;
        s_mask[j] = njobs ? __ldcg(f.mask + j) : 0;
    }
    __syncthreads();
    struct Item {
        Rows16 w;
        int job, b, mask;
        float sw;
    };
    auto load = [&](Item (&q)[kBatch], int first) {
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            const int i = first + u * kWarps;
            const bool in = i < items;
            q[u].job = in ? i / fb : 0;
            q[u].b = in ? i - q[u].job * fb : 0;
            const int64_t e = s_expert[q[u].job];
            q[u].mask = in ? s_mask[q[u].job] : 0;
            q[u].sw = __ldg(a.w.d_down_s + (e * sblocks(H) + n0 / kSBlk) * fb + q[u].b);
            q[u].w.load(a.w.d_down + (e * H + n0 + g) * F, F, in, q[u].b * kSBlk + 16 * tig, F);
        }
    };
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto batch = [&](Item (&q)[kBatch], Item (&n)[kBatch], int first) {
        // the activations first: a wait for them must not wait for the next weights
        uint4 x0[kBatch], x1[kBatch];
        float s[kBatch][2];
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            const int64_t row = (int64_t)q[u].job * kSmallT;
            const int k0 = q[u].b * kSBlk + 16 * tig;
            const bool col = (q[u].mask >> g) & 1;
            const uint8_t *hr = f.hq + (row + g) * F;
            x0[u] = ldcg16_if(hr + k0, col && k0 < F);
            x1[u] = ldcg16_if(hr + k0 + 64, col && k0 + 64 < F);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const bool on = (q[u].mask >> (2 * tig + c)) & 1;
                s[u][c] = on ? __ldcg(f.hs + (row + 2 * tig + c) * fb + q[u].b) *
                                   __ldcg(f.weight + row + 2 * tig + c)
                             : 0.f;
            }
        }
        load(n, first + kBatch * kWarps);
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            if (!q[u].mask) continue;
            float cc[4] = {0.f, 0.f, 0.f, 0.f};
            q[u].w.multiply(cc, x0[u], x1[u]);
            // a token that is not routed here takes nothing, whatever the weights hold
#pragma unroll
            for (int c = 0; c < 2; c++) {
                if (!((q[u].mask >> (2 * tig + c)) & 1)) continue;
                acc[c] = fmaf(cc[c], s[u][c] * q[u].sw, acc[c]);
                acc[c + 2] = fmaf(cc[c + 2], s[u][c] * q[u].sw, acc[c + 2]);
            }
        }
    };
    Item q0[kBatch], q1[kBatch];
    load(q0, warp);
    ptx::grid_dependency_wait();
    for (int first = warp; first < items; first += 2 * kBatch * kWarps) {
        batch(q0, q1, first);
        if (first + kBatch * kWarps >= items) break;
        batch(q1, q0, first + kBatch * kWarps);
    }
    put_frag(red[warp], acc, g, tig);
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kTile * 8 && i / kTile < a.T) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) sum += red[w][i];
        static_cast<T *>(a.out)[(int64_t)(i / kTile) * H + n0 + i % kTile] = from_f32<T>(sum);
    }
}

}  // namespace

cudaError_t launch_scaled_small(const ScaledMatmulArgs &a, cudaStream_t st) {
    if (a.M <= 0) return cudaSuccess;
    if (a.M > kSmallT) return cudaErrorInvalidValue;
    const unsigned grid = (a.N + kTile - 1) / kTile;
    return with_dtype(a.dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        k_scaled_rows<E><<<grid, kWarps * 32, 0, st>>>(a);
        note_launches(1);
        return cudaGetLastError();
    });
}

size_t scaled_small_ws_bytes(int T, int k, int shared, int H, int F) {
    const size_t one = (size_t)(k + shared) * F * sizeof(float);
    return T == 1 ? one : std::max(one, few_layout(T, k, shared, H, F, nullptr, nullptr));
}

cudaError_t launch_scaled_experts_small(const ScaledExpertsArgs &e, void *ws, cudaStream_t st) {
    ScaledExpertsArgs a = e;
    const int jobs = a.T * a.k + a.w.shared;
    if (a.T == 1) {
        a.h = static_cast<float *>(ws);
        const cudaError_t err = with_dtype(a.x_dt, [&](auto *tag) {
            using E = std::remove_pointer_t<decltype(tag)>;
            k_one_gateup<E><<<dim3(a.w.ffn / kTile, jobs), kWarps * 32, 0, st>>>(a);
            note_launches(1);
            return cudaGetLastError();
        });
        if (err != cudaSuccess) return err;
        return with_dtype(a.out_dt, [&](auto *tag) {
            using E = std::remove_pointer_t<decltype(tag)>;
            return launch_behind(k_one_down<E>, dim3(a.w.hidden / kTile), kWarps * 32, 0, st, a);
        });
    }
    FewWs f;
    few_layout(a.T, a.k, a.w.shared, a.w.hidden, a.w.ffn, static_cast<uint8_t *>(ws), &f);
    cudaError_t err = with_dtype(a.x_dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const int units = a.T * sblocks(a.w.hidden);
        k_few_prep<E><<<1 + (units + 7) / 8, 256, 0, st>>>(a, f);
        note_launches(1);
        return cudaGetLastError();
    });
    if (err != cudaSuccess) return err;
    err = launch_behind(k_few_gateup, dim3(sblocks(a.w.ffn), jobs), kFewThreads, 0, st, a, f);
    if (err != cudaSuccess) return err;
    return with_dtype(a.out_dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        return launch_behind(k_few_down<E>, dim3(a.w.hidden / kTile), kWarps * 32, 0, st, a, f);
    });
}

}  // namespace moe
