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
// The weights of 16 rows are split over k among a CTA's 8 warps; their partial sums meet in
// shared memory in the order of the warps, so results repeat.
#include "ptx.cuh"
#include "scaled.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;                 // weight rows per CTA
constexpr int kPitch = kSBlk + 16;        // bytes per activation row in shared memory

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

__device__ __forceinline__ uint4 ldg_stream(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
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

// 16 bytes of row p at column k of K columns, zeros past the end (the row's stride is a multiple
// of 16, so a chunk that starts inside it lies inside it).
__device__ __forceinline__ uint4 row16(const uint8_t *p, int k, int K) {
    if (!p || k >= K) return make_uint4(0u, 0u, 0u, 0u);
    const uint4 v = ldg_stream(p + k);
    return K - k >= 16 ? v : keep_bytes(v, K - k);
}

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

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_scaled_rows(const ScaledMatmulArgs a) {
    __shared__ float red[kWarps][kTile * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int n0 = blockIdx.x * kTile, m0 = blockIdx.y * 8;
    const int nb = sblocks(a.K);
    const uint8_t *lo = n0 + g < a.N ? a.b + (int64_t)(n0 + g) * a.ldb : nullptr;
    const uint8_t *hi = n0 + g + 8 < a.N ? a.b + (int64_t)(n0 + g + 8) * a.ldb : nullptr;
    const uint8_t *xr = m0 + g < a.M ? a.a + (int64_t)(m0 + g) * a.lda : nullptr;
    const float *ws = a.bs + (int64_t)(n0 / kSBlk) * nb;
    const int c0 = m0 + 2 * tig, c1 = c0 + 1;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b = warp; b < nb; b += kWarps) {
        const int k0 = b * kSBlk + 16 * tig;
        const uint4 l0 = row16(lo, k0, a.K), l1 = row16(lo, k0 + 64, a.K);
        const uint4 h0 = row16(hi, k0, a.K), h1 = row16(hi, k0 + 64, a.K);
        const uint4 x0 = row16(xr, k0, a.K), x1 = row16(xr, k0 + 64, a.K);
        const float sw = __ldg(ws + b);
        const float s0 = c0 < a.M ? __ldg(a.as + b * a.ldas + c0) * sw : 0.f;
        const float s1 = c1 < a.M ? __ldg(a.as + b * a.ldas + c1) * sw : 0.f;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma64(c, l0, h0, x0);
        mma64(c, l1, h1, x1);
        acc[0] = fmaf(c[0], s0, acc[0]);
        acc[1] = fmaf(c[1], s1, acc[1]);
        acc[2] = fmaf(c[2], s0, acc[2]);
        acc[3] = fmaf(c[3], s1, acc[3]);
    }
    put_frag(red[warp], acc, g, tig);
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kTile * 8) {
        const int m = m0 + i / kTile, n = n0 + i % kTile;
        if (m < a.M && n < a.N)
            static_cast<T *>(a.out)[m * a.ldo + n] = from_f32<T>(sum_warps(red, i));
    }
}

// ------------------------------------------------------------------ the experts

// The distinct experts of the batch, in order of first appearance in ids, then the shared one:
// job j's expert, and per token the weight of its output (the sum over the token's slots that
// name the expert) with a bit telling whether it is routed there at all.  All threads of the CTA;
// s_ids holds T * k entries, at most one per thread.
struct Jobs {
    int n;
    int expert[kSmallT * kMaxK + 1];
    int count[kWarps + 1];
};

__device__ __forceinline__ void build_jobs(const ScaledExpertsArgs &a, Jobs &J, int *s_ids) {
    const int A = a.T * a.k, i = threadIdx.x, lane = i & 31, warp = i >> 5;
    int e = -1;
    if (i < A) {
        e = a.ids[i];
        if (e < 0 || e >= a.w.n_experts) {
            e = -1;
            set_status(a.status, MOE_ERR_BOUNDS);
        }
        s_ids[i] = e;
    }
    __syncthreads();
    bool first = i < A && e >= 0;
    for (int b = 0; b < i && first; b++) first = s_ids[b] != e;
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (lane == 0) J.count[warp] = __popc(m);
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        base += w < warp ? J.count[w] : 0;
        total += J.count[w];
    }
    if (first) J.expert[base + __popc(m & ((1u << lane) - 1u))] = e;
    if (i == 0) {
        if (a.w.shared) J.expert[total] = a.w.n_experts;
        J.n = total + (a.w.shared ? 1 : 0);
    }
    __syncthreads();
}

// Whether token t is routed to expert e, and with what weight.
__device__ __forceinline__ bool routed(const ScaledExpertsArgs &a, const int *s_ids, int e, int t,
                                       float *w) {
    if (e == a.w.n_experts) {
        *w = a.gate ? a.gate[t] : 1.0f;
        return true;
    }
    bool on = false;
    float s = 0.f;
    for (int j = 0; j < a.k; j++) {
        if (s_ids[t * a.k + j] != e) continue;
        on = true;
        s += a.rw[t * a.k + j];
    }
    *w = s;
    return on;
}

// Activation columns of one block for a warp: 8 rows of e4m3 bytes and their scales.
struct __align__(16) Cols {
    uint8_t q[8 * kPitch];
    float s[8];
};

__device__ __forceinline__ void put_col(Cols &C, int t, float4 v, uint32_t *status) {
    const int lane = threadIdx.x & 31;
    float s;
    bool fin;
    const uint32_t p = quant_block(v, &s, &fin);
    *reinterpret_cast<uint32_t *>(C.q + t * kPitch + 4 * lane) = p;
    if (lane == 0) {
        C.s[t] = s;
        if (!fin) set_status(status, MOE_ERR_NONFINITE);
    }
}

// grid (ffn / 16, most jobs): h of 16 rows of one job's expert for the tokens routed to it.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_small_gateup(const ScaledExpertsArgs a) {
    __shared__ float red[2][kWarps][kTile * 8];
    __shared__ Cols cols[kWarps];
    __shared__ Jobs J;
    __shared__ int s_ids[kSmallT * kMaxK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    ptx::launch_dependents();
    for (int i = threadIdx.x; i < kWarps * (int)sizeof(Cols) / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(cols)[i] = 0u;
    build_jobs(a, J, s_ids);
    const int j = blockIdx.y;
    if (j >= J.n) return;
    const int e = J.expert[j];
    const int H = a.w.hidden, F = a.w.ffn, hb = sblocks(H);
    const int f0 = blockIdx.x * kTile;
    const int64_t r0 = (int64_t)e * F + f0;
    const uint8_t *wg = a.w.d_gate + r0 * H, *wu = a.w.d_up + r0 * H;
    const int64_t sb = ((int64_t)e * sblocks(F) + f0 / kSBlk) * hb;
    const float *gs = a.w.d_gate_s + sb, *us = a.w.d_up_s + sb;
    unsigned on = 0;
    for (int t = 0; t < a.T; t++) {
        float w;
        if (routed(a, s_ids, e, t, &w)) on |= 1u << t;
    }
    Cols &C = cols[warp];
    float ag[4] = {0.f, 0.f, 0.f, 0.f}, au[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b = warp; b < hb; b += kWarps) {
        const int k0 = b * kSBlk + 16 * tig;
        const uint8_t *g0 = wg + (int64_t)g * H, *g1 = g0 + 8 * (int64_t)H;
        const uint8_t *u0 = wu + (int64_t)g * H, *u1 = u0 + 8 * (int64_t)H;
        const uint4 w0 = row16(g0, k0, H), w1 = row16(g1, k0, H);
        const uint4 w2 = row16(g0, k0 + 64, H), w3 = row16(g1, k0 + 64, H);
        const uint4 v0 = row16(u0, k0, H), v1 = row16(u1, k0, H);
        const uint4 v2 = row16(u0, k0 + 64, H), v3 = row16(u1, k0 + 64, H);
        const float sg = __ldg(gs + b), su = __ldg(us + b);
        const int c = b * kSBlk + 4 * lane;
        for (int t = 0; t < a.T; t++) {
            if (!((on >> t) & 1u)) continue;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < H) v = load4(static_cast<const T *>(a.x) + (int64_t)t * H + c);
            put_col(C, t, v, a.status);
        }
        __syncwarp();
        const uint4 x0 = *reinterpret_cast<const uint4 *>(C.q + g * kPitch + 16 * tig);
        const uint4 x1 = *reinterpret_cast<const uint4 *>(C.q + g * kPitch + 64 + 16 * tig);
        const float s0 = C.s[2 * tig], s1 = C.s[2 * tig + 1];
        float cg[4] = {0.f, 0.f, 0.f, 0.f}, cu[4] = {0.f, 0.f, 0.f, 0.f};
        mma64(cg, w0, w1, x0);
        mma64(cu, v0, v1, x0);
        mma64(cg, w2, w3, x1);
        mma64(cu, v2, v3, x1);
        ag[0] = fmaf(cg[0], s0 * sg, ag[0]);
        ag[1] = fmaf(cg[1], s1 * sg, ag[1]);
        ag[2] = fmaf(cg[2], s0 * sg, ag[2]);
        ag[3] = fmaf(cg[3], s1 * sg, ag[3]);
        au[0] = fmaf(cu[0], s0 * su, au[0]);
        au[1] = fmaf(cu[1], s1 * su, au[1]);
        au[2] = fmaf(cu[2], s0 * su, au[2]);
        au[3] = fmaf(cu[3], s1 * su, au[3]);
        __syncwarp();
    }
    put_frag(red[0][warp], ag, g, tig);
    put_frag(red[1][warp], au, g, tig);
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kTile * 8 && ((on >> (i / kTile)) & 1u)) {
        const float gv = sum_warps(red[0], i), uv = sum_warps(red[1], i);
        a.h[((int64_t)j * kSmallT + i / kTile) * F + f0 + i % kTile] =
            __fdiv_rn(gv, 1.0f + expf(-gv)) * uv;
    }
}

// grid (hidden / 16): 16 output rows for all tokens, over every job.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_small_down(const ScaledExpertsArgs a) {
    __shared__ float red[kWarps][kTile * 8];
    __shared__ Cols cols[kWarps];
    __shared__ Jobs J;
    __shared__ int s_ids[kSmallT * kMaxK];
    __shared__ float s_w[kSmallT * kMaxK + 1][kSmallT];
    __shared__ uint8_t s_on[kSmallT * kMaxK + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    for (int i = threadIdx.x; i < kWarps * (int)sizeof(Cols) / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(cols)[i] = 0u;
    build_jobs(a, J, s_ids);
    for (int j = threadIdx.x; j < J.n; j += blockDim.x) {
        unsigned on = 0;
        for (int t = 0; t < a.T; t++) {
            float w;
            if (routed(a, s_ids, J.expert[j], t, &w)) on |= 1u << t;
            s_w[j][t] = w;
        }
        for (int t = a.T; t < kSmallT; t++) s_w[j][t] = 0.f;
        s_on[j] = (uint8_t)on;
    }
    __syncthreads();
    const int H = a.w.hidden, F = a.w.ffn, fb = sblocks(F);
    const int n0 = blockIdx.x * kTile;
    Cols &C = cols[warp];
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    ptx::grid_dependency_wait();
    for (int i = warp; i < J.n * fb; i += kWarps) {
        const int j = i / fb, b = i - j * fb, e = J.expert[j];
        const unsigned on = s_on[j];
        const uint8_t *p0 = a.w.d_down + ((int64_t)e * H + n0 + g) * F, *p1 = p0 + 8 * (int64_t)F;
        const int k0 = b * kSBlk + 16 * tig;
        const uint4 w0 = row16(p0, k0, F), w1 = row16(p1, k0, F);
        const uint4 w2 = row16(p0, k0 + 64, F), w3 = row16(p1, k0 + 64, F);
        const float sw = __ldg(a.w.d_down_s + ((int64_t)e * sblocks(H) + n0 / kSBlk) * fb + b);
        const int c = b * kSBlk + 4 * lane;
        for (int t = 0; t < a.T; t++) {
            if (!((on >> t) & 1u)) continue;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < F)
                v = __ldcg(reinterpret_cast<const float4 *>(
                    a.h + ((int64_t)j * kSmallT + t) * F + c));
            put_col(C, t, v, a.status);
        }
        __syncwarp();
        const uint4 x0 = *reinterpret_cast<const uint4 *>(C.q + g * kPitch + 16 * tig);
        const uint4 x1 = *reinterpret_cast<const uint4 *>(C.q + g * kPitch + 64 + 16 * tig);
        float cc[4] = {0.f, 0.f, 0.f, 0.f};
        mma64(cc, w0, w1, x0);
        mma64(cc, w2, w3, x1);
        // a token that is not routed here takes nothing, whatever its column holds
        if ((on >> (2 * tig)) & 1u) {
            const float s = C.s[2 * tig] * sw;
            const float r = s_w[j][2 * tig];
            acc[0] = fmaf(cc[0] * s, r, acc[0]);
            acc[2] = fmaf(cc[2] * s, r, acc[2]);
        }
        if ((on >> (2 * tig + 1)) & 1u) {
            const float s = C.s[2 * tig + 1] * sw;
            const float r = s_w[j][2 * tig + 1];
            acc[1] = fmaf(cc[1] * s, r, acc[1]);
            acc[3] = fmaf(cc[3] * s, r, acc[3]);
        }
        __syncwarp();
    }
    put_frag(red[warp], acc, g, tig);
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kTile * 8 && i / kTile < a.T)
        static_cast<T *>(a.out)[(int64_t)(i / kTile) * H + n0 + i % kTile] =
            from_f32<T>(sum_warps(red, i));
}

}  // namespace

cudaError_t launch_scaled_small(const ScaledMatmulArgs &a, cudaStream_t st) {
    if (a.M <= 0) return cudaSuccess;
    const dim3 grid((a.N + kTile - 1) / kTile, (a.M + 7) / 8);
    return with_dtype(a.dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        k_scaled_rows<E><<<grid, kWarps * 32, 0, st>>>(a);
        note_launches(1);
        return cudaGetLastError();
    });
}

size_t scaled_small_h_bytes(int T, int k, int shared, int F) {
    return (size_t)(T * k + (shared ? 1 : 0)) * kSmallT * F * sizeof(float);
}

cudaError_t launch_scaled_experts_small(const ScaledExpertsArgs &a, cudaStream_t st) {
    const dim3 grid(a.w.ffn / kTile, a.T * a.k + (a.w.shared ? 1 : 0));
    cudaError_t err = with_dtype(a.x_dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        k_small_gateup<E><<<grid, kWarps * 32, 0, st>>>(a);
        note_launches(1);
        return cudaGetLastError();
    });
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.w.hidden / kTile);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return with_dtype(a.out_dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const cudaError_t r = cudaLaunchKernelEx(&cfg, k_small_down<E>, a);
        if (r != cudaSuccess) return r;
        note_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace moe
