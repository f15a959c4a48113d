// k_scaled_quant.cu -- activations to e4m3 with one fp32 scale per row and 128 columns.
//
// Reads every value once and writes a byte per value and 4 bytes per 128: bound by memory.  A
// warp takes four rows of one column block, so that four loads are in flight per lane and the
// four scales, neighbours in the block-major scale array, go out together.
#include "route_dev.cuh"
#include "scaled.cuh"

namespace moe {

namespace {

constexpr int kRows = 4;       // rows per warp
constexpr int kThreads = 256;

// Where the bytes and scales of row t go: row t itself, or every slot of token t.
struct Rows {
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t lds;
    static constexpr bool kList = false;
    __device__ __forceinline__ int count() const { return 1; }
    __device__ __forceinline__ int64_t row(int64_t t, int, uint32_t *) const { return t; }
};
struct Slots {
    SliceArgs slices;             // listed by one more CTA
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t lds;
    const int32_t *inv_perm;
    int k, routed, shared;
    static constexpr bool kList = true;
    __device__ __forceinline__ int count() const { return k + shared; }
    __device__ __forceinline__ int64_t row(int64_t t, int j, uint32_t *status) const {
        if (j == k) return routed + t;
        const int p = __ldg(inv_perm + t * k + j);
        if (p >= 0 && p < routed) return p;
        set_status(status, MOE_ERR_BOUNDS);
        return -1;
    }
};

// The runs of up to kScaledRun slots of every expert with tokens, ascending, the shared one's
// last.  One CTA.
__device__ void list_slices(const SliceArgs &a, uint32_t *status) {
    __shared__ int s_first[kMaxE];
    __shared__ int s_warp[33];
    const int A = a.T * a.k;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const int o = a.offsets[e], o1 = a.offsets[e + 1];
        const bool fits = o >= 0 && o <= o1 && o1 <= A;      // else not what a router wrote
        if (!fits) set_status(status, MOE_ERR_BOUNDS);
        s_first[e] = fits ? (o1 - o + kScaledRun - 1) / kScaledRun : 0;
    }
    __syncthreads();
    // overlapping runs of damaged offsets could pass the list's end: those are left out too
    const int most = A / kScaledRun + min(a.E, A);
    const int n = min(block_exclusive_scan<kThreads>(s_first, a.E, s_warp), most);
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const int o = a.offsets[e], o1 = a.offsets[e + 1];
        if (!(o >= 0 && o <= o1 && o1 <= A)) continue;
        for (int s = o, j = s_first[e]; s < o1 && j < most; s += kScaledRun, j++)
            a.slices[j] = Job{e, s, min(kScaledRun, o1 - s), 0};
    }
    const int ns = a.shared ? (a.T + kScaledRun - 1) / kScaledRun : 0;
    for (int j = threadIdx.x; j < ns; j += kThreads)
        a.slices[n + j] = Job{a.E, A + j * kScaledRun, min(kScaledRun, a.T - j * kScaledRun), 1};
    if (threadIdx.x == 0) *a.nslices = n + ns;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load_rows(const T *x, int64_t t0, int c, int rows, int K,
                                          int64_t ldx, float4 (&v)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + i >= rows) continue;
        const T *p = x + (t0 + i) * ldx + c;
        if (kVec) {
            if (c < K) v[i] = load4(p);
        } else {
            if (c < K) v[i].x = to_f32(p[0]);
            if (c + 1 < K) v[i].y = to_f32(p[1]);
            if (c + 2 < K) v[i].z = to_f32(p[2]);
            if (c + 3 < K) v[i].w = to_f32(p[3]);
        }
    }
}

template <typename T, bool kVec, typename To>
__global__ void __launch_bounds__(kThreads)
    k_scaled_quantize(const T *__restrict__ x, int rows, int K, int64_t ldx, const To to,
                      uint32_t *status) {
    int cta = blockIdx.x;
    if constexpr (To::kList) {             // the first CTA: its work is the longest
        if (cta-- == 0) {
            list_slices(to.slices, status);
            return;
        }
    }
    const int lane = threadIdx.x & 31;
    const int nb = sblocks(K);
    const int64_t unit = (int64_t)cta * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t rt = unit / nb;
    const int b = (int)(unit - rt * nb);
    const int64_t t0 = rt * kRows;
    if (t0 >= rows) return;
    const int c = b * kSBlk + lane * 4;
    float4 v[kRows];
    load_rows<T, kVec>(x, t0, c, rows, K, ldx, v);
    // the largest magnitudes as integers (a NaN or an infinity has the largest bit patterns);
    // lane i takes row i's scale and reciprocal, one division for the four
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits(v[i]));
        if (lane == i) top = m;
    }
    const bool bad = top >= 0x7f800000u;
    const float sc = bad ? 0.f : __fdiv_rn(__uint_as_float(top), kE4M3Max);
    const float inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
    if (bad) set_status(status, MOE_ERR_NONFINITE);
    uint32_t p[kRows];
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const float s = __shfl_sync(0xffffffffu, sc, i), r = __shfl_sync(0xffffffffu, inv, i);
        p[i] = s > 0.f ? quant4(v[i], s, r) : 0u;
    }
    for (int j = 0; j < to.count(); j++) {
        int64_t at = -1;
        if (lane < kRows && t0 + lane < rows) {
            at = to.row(t0 + lane, j, status);
            if (at >= 0) to.s[b * to.lds + at] = sc;
        }
#pragma unroll
        for (int i = 0; i < kRows; i++) {
            const int64_t r = __shfl_sync(0xffffffffu, at, i);
            if (r < 0) continue;
            uint8_t *o = to.q + r * to.ldq + c;
            if (c + 3 < K) {
                *reinterpret_cast<uint32_t *>(o) = p[i];
            } else {
                for (int n = 0; n < 3; n++)
                    if (c + n < K) o[n] = (uint8_t)(p[i] >> (8 * n));
            }
        }
    }
}

template <typename To>
cudaError_t run(const void *x, int dt, int T, int K, int64_t ldx, const To &to, uint32_t *status,
                cudaStream_t st) {
    if (T <= 0) return cudaSuccess;
    const int64_t units = (int64_t)((T + kRows - 1) / kRows) * sblocks(K);
    const unsigned grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)) + To::kList;
    return with_dtype(dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const E *p = static_cast<const E *>(x);
        // vector loads where every lane's four elements start on their natural boundary
        const bool vec = ((uintptr_t)x % (4 * sizeof(E))) == 0 && ldx % 4 == 0 && K % 4 == 0;
        if (vec)
            k_scaled_quantize<E, true, To><<<grid, kThreads, 0, st>>>(p, T, K, ldx, to, status);
        else
            k_scaled_quantize<E, false, To><<<grid, kThreads, 0, st>>>(p, T, K, ldx, to, status);
        note_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_scaled_quantize(const void *x, int dt, int T, int K, int64_t ldx, uint8_t *q,
                                   int64_t ldq, float *s, int64_t lds, uint32_t *status,
                                   cudaStream_t st) {
    return run(x, dt, T, K, ldx, Rows{q, ldq, s, lds}, status, st);
}

cudaError_t launch_scaled_spread(const ScaledExpertsArgs &e, uint8_t *q, float *s, Job *slices,
                                 int32_t *nslices, cudaStream_t st) {
    const int A = e.T * e.k;
    const Slots to{{e.offsets, e.w.n_experts, e.T, e.k, e.w.shared, slices, nslices},
                   q, e.w.hidden, s, (int64_t)A + (e.w.shared ? e.T : 0), e.inv_perm, e.k, A,
                   e.w.shared};
    return run(e.x, e.x_dt, e.T, e.w.hidden, e.w.hidden, to, e.status, st);
}

}  // namespace moe
