// k_scaled_quant.cu -- activations to e4m3 with one fp32 scale per row and 128 columns.
//
// Reads every value once and writes a byte per value and 4 bytes per 128.  16-bit rows are bound by
// instructions before memory, so the work is laid out to need few: a half warp holds a block, 8
// values per lane in one 16-byte load, so that its 16 lanes all end up with the block's largest
// magnitude after four shuffles and take the division without passing it around; 16-bit
// magnitudes are compared two at a time.  A warp takes four rows of two neighbouring blocks, so
// that four loads are in flight and the scales of four rows, neighbours in the block-major scale
// array, go out together.  8192 x 2560 bf16: 18.3 to 20.7 us on the device (22 instructions a value, half of
// them for near-ties, 71 % of the issue slots), fp16 16.7, fp32 22.7 us; 3 rows 2.8 us.
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

__device__ __forceinline__ float4 widen4(uint32_t a, uint32_t b, __nv_bfloat16 *) {
    return make_float4(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u),
                       __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}
__device__ __forceinline__ float4 widen4(uint32_t a, uint32_t b, __half *) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    return make_float4(x.x, x.y, y.x, y.y);
}

// Eight consecutive values of a row as they came.
template <typename T>
struct Eight {                          // 16-bit types, two per word
    uint32_t w[4];
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void load(const T *p) {
        const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
    }
    __device__ __forceinline__ void load(const T *p, int n) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n)
                w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << (16 * (i & 1));
    }
    __device__ __forceinline__ float4 quad(int i) const { return widen4(w[2 * i], w[2 * i + 1], (T *)nullptr); }
    // the largest magnitude as an fp32 pattern (an infinity or NaN has the largest ones)
    __device__ __forceinline__ uint32_t largest() const {
        const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                    __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        const uint16_t h = (uint16_t)max(m & 0xffffu, m >> 16);
        return __float_as_uint(to_f32(*reinterpret_cast<const T *>(&h)));
    }
};
template <>
struct Eight<float> {
    float f[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = 0.f;
    }
    __device__ __forceinline__ void load(const float *p) {
        const float4 a = load4(p), b = load4(p + 4);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void load(const float *p, int n) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) f[i] = p[i];
    }
    __device__ __forceinline__ float4 quad(int i) const {
        return make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    }
    __device__ __forceinline__ uint32_t largest() const {
        return max(abs_bits(make_float4(f[0], f[1], f[2], f[3])),
                   abs_bits(make_float4(f[4], f[5], f[6], f[7])));
    }
};

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
    const uint32_t pairs = ((uint32_t)sblocks(K) + 1) / 2;
    const uint32_t unit = (uint32_t)cta * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t rt = unit / pairs, pr = unit - rt * pairs;
    const int64_t t0 = (int64_t)rt * kRows;
    if (t0 >= rows) return;
    const int b = 2 * (int)pr + (lane >> 4), c = 2 * (int)pr * kSBlk + lane * 8;
    Eight<T> v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        v[i].clear();
        if (t0 + i >= rows || c >= K) continue;
        const T *p = x + (t0 + i) * ldx + c;
        if (kVec)
            v[i].load(p);
        else
            v[i].load(p, K - c);
    }
    float sc[kRows];
    uint2 q[kRows];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        uint32_t top = v[i].largest();
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        sc[i] = scale_of(top);
        bad = bad || top >= 0x7f800000u;
        float inv;                     // 1 / scale within 2^-23, inf for 0
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sc[i]));
        const float below = inv * kBelow, above = inv * kAbove;
        const float4 a = v[i].quad(0), d = v[i].quad(1);
        q[i] = make_uint2(quant4_at(a, below), quant4_at(d, below));
        const uint2 hi = make_uint2(quant4_at(a, above), quant4_at(d, above));
        if (sc[i] < 0x1p-100f) {       // zero, not finite, or too small for the arithmetic below
            q[i] = sc[i] > 0.f ? make_uint2(quant4_wide(a, sc[i]), quant4_wide(d, sc[i]))
                               : make_uint2(0u, 0u);
        } else if (q[i].x != hi.x || q[i].y != hi.y) {
            // halfway or close, decided one by one: one bf16 value in 194, in a quarter of the blocks
            // (they come together, where the scale has few bits); one fp16 value in 1600, one fp32
            // value in 87000 (N(0, 1), one channel in a hundred 20 times larger)
            const float f[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
#pragma unroll 1
            for (uint32_t x = q[i].x ^ hi.x, y = q[i].y ^ hi.y; x | y;) {
                const int n = x ? (__ffs(x) - 1) >> 3 : 4 + ((__ffs(y) - 1) >> 3);
                float val = f[0];
#pragma unroll
                for (int e = 1; e < 8; e++) val = n == e ? f[e] : val;
                const uint32_t shift = 8 * (n & 3), mask = 0xffu << shift;
                const uint32_t l = ((n < 4 ? q[i].x : q[i].y) >> shift) & 0xffu;
                const uint32_t h = ((n < 4 ? hi.x : hi.y) >> shift) & 0xffu;
                const uint32_t c8 = quant1_decide(val, sc[i], l, h) << shift;
                if (n < 4) {
                    q[i].x = (q[i].x & ~mask) | c8;
                    x &= ~mask;
                } else {
                    q[i].y = (q[i].y & ~mask) | c8;
                    y &= ~mask;
                }
            }
        }
    }
    if (bad) set_status(status, MOE_ERR_NONFINITE);
    // lane 16 h + i holds the scale of row i, block h
    float mine = sc[0];
#pragma unroll
    for (int i = 1; i < kRows; i++) mine = (lane & 15) == i ? sc[i] : mine;
    const bool scale_lane = (lane & 15) < kRows && t0 + (lane & 15) < rows;
    for (int j = 0; j < to.count(); j++) {
        int64_t at = -1;
        if (scale_lane) {
            at = to.row(t0 + (lane & 15), j, status);
            if (at >= 0 && b * kSBlk < K) to.s[b * to.lds + at] = mine;
        }
#pragma unroll
        for (int i = 0; i < kRows; i++) {
            int64_t r;
            if constexpr (To::kList)
                r = __shfl_sync(0xffffffffu, at, i);
            else
                r = t0 + i < rows ? t0 + i : -1;
            if (r < 0 || c >= K) continue;
            uint8_t *o = to.q + r * to.ldq + c;
            if (c + 8 <= K) {
                *reinterpret_cast<uint2 *>(o) = q[i];
            } else {
                for (int n = 0; n < 7; n++)
                    if (c + n < K) o[n] = (uint8_t)((n < 4 ? q[i].x : q[i].y) >> (8 * (n & 3)));
            }
        }
    }
}

template <typename To>
cudaError_t run(const void *x, int dt, int T, int K, int64_t ldx, const To &to, uint32_t *status,
                cudaStream_t st) {
    if (T <= 0) return cudaSuccess;
    const int64_t units = (int64_t)((T + kRows - 1) / kRows) * ((sblocks(K) + 1) / 2);
    const unsigned grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)) + To::kList;
    return with_dtype(dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const E *p = static_cast<const E *>(x);
        // vector loads where every lane's eight elements start on a 16-byte boundary
        const bool vec = (uintptr_t)x % 16 == 0 && ldx * sizeof(E) % 16 == 0 && K % 8 == 0;
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
