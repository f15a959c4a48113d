// scaled.cuh -- shared declarations of the float8 (e4m3, 128-block scaled) operators: element
// types, the quantiser of one block, and the launchers behind the moe_scaled_* entry points.
#pragma once

#include <cuda_bf16.h>

#include "moe_internal.cuh"

namespace moe {

constexpr int kSBlk = 128;                 // columns (and weight rows) per scale
constexpr float kE4M3Max = 448.0f;
// Most rows of the product's small kernel: the columns of one MMA.  Caches cold, small kernel /
// tensor cores: 8 rows of 1280 x 2560 weights 8.2 / 14.3 us, of 1280 x 8192 14.3 / 28.7, of
// 8192 x 8192 24.6 / 34.8.  More rows would read the weights once per eight: 9 rows of the same
// 10.2 / 14.3, 14.4 / 28.7 and 36.9 / 34.8 us, better for few weight rows and worse for many; that
// form is not kept.
constexpr int kSmallT = 8;
// Most tokens of the experts' small-batch kernels.  Caches cold, every expert equally likely, with a
// shared one, small / tensor cores at 2, 4, 5 and 8 tokens: 10 of 512 experts (hidden 2560, ffn 640)
// 45 / 55, 74 / 78, 84 / 84, 121 / 107 us; 6 of 64 (2048, 512) 31 / 39, 39 / 45, 45 / 47, 53 / 53; 2 of
// 8 (2048, 512) 25 / 33, 29 / 35, 29 / 35, 31 / 35.  What moves the crossover is the number of
// distinct experts; a rule in tokens alone gives up to a sixth away at 5 to 8 tokens of few experts.
constexpr int kSmallExpertsT = 4;

__host__ __device__ inline int sblocks(int n) { return (n + kSBlk - 1) / kSBlk; }
inline size_t dtype_bytes(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }
inline bool dtype_ok(int dt) { return dt >= MOE_DT_F32 && dt <= MOE_DT_F16; }

// One call of f with a null pointer of the element type of `dt` (the type is what matters).
template <typename F>
inline cudaError_t with_dtype(int dt, F &&f) {
    switch (dt) {
        case MOE_DT_F32: return f((float *)nullptr);
        case MOE_DT_BF16: return f((__nv_bfloat16 *)nullptr);
        default: return f((__half *)nullptr);
    }
}

// ------------------------------------------------------------------ element types

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Four consecutive elements at p (16-byte aligned for fp32, 8-byte for the 16-bit types).
__device__ __forceinline__ float4 load4(const float *p) {
    return __ldg(reinterpret_cast<const float4 *>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 load4(const __half *p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&r.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

// ------------------------------------------------------------------ e4m3 of one block

// Two values to two e4m3 bytes (lo in the low byte), nearest, ties to even, clamped to +-448.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// x / s to the nearest e4m3 without an intermediate rounding, for any s > 0: the 64-bit quotient,
// rounded to fp32 with its lost bits kept as a sticky last bit, converts as the exact quotient
// would (fp32 has 20 bits more than e4m3, and a 64-bit quotient of two fp32 values is never
// halfway between two e4m3 values unless it is exact).
static __device__ __noinline__ uint32_t quant4_wide(float4 v, float s) {
    float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const double q = __ddiv_rn((double)f[i], (double)s);
        float r = __double2float_rz(q);
        if ((double)r != q) r = __uint_as_float(__float_as_uint(r) | 1u);
        f[i] = r;
    }
    return cvt_e4m3x2(f[0], f[1]) | (cvt_e4m3x2(f[2], f[3]) << 16);
}

// The scale amax / 448 of a largest magnitude given as an fp32 pattern, 0 when it is not finite.  A
// product with 1 / 448, its exact remainder and one more multiply-add give the correctly rounded
// quotient (P. Markstein's correction of a quotient by its remainder); near the subnormals, where the remainder may underflow, the division does.
__device__ __forceinline__ float scale_of(uint32_t top) {
    const float x = __uint_as_float(top);
    constexpr float r = 1.0f / kE4M3Max;
    const float q = x * r;
    const float s = fmaf(fmaf(-q, kE4M3Max, x), r, q);
    if (top >= 0x7f800000u) return 0.f;
    return x < 0x1p-90f ? __fdiv_rn(x, kE4M3Max) : s;
}

// v / s to e4m3 where it lies between the neighbouring codes l and h (of v's sign, |l| < |h|): v is
// compared with s times the value halfway between them, exactly, in one multiply-add; equal goes
// to the even code.
__device__ __forceinline__ uint32_t quant1_decide(float v, float s, uint32_t l, uint32_t h) {
    uint32_t x;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(l | (h << 8))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
    const float r = fmaf(-0.5f * fabsf(f.x + f.y), s, fabsf(v));      // the sum and half are exact
    return r > 0.f || (r == 0.f && (l & 1u)) ? h : l;
}

// Four values of a block with scale s > 0 as packed e4m3.  v / s by a reciprocal within 2^-23 of
// 1 / s is within 2^-21; when the values 2^-21 below and above it convert to the same byte, so
// does v / s (conversion is monotone).  Otherwise they are neighbours and quant1_decide tells.
// 16-bit inputs are halfway often (their quotients have few bits), so this costs no division.
constexpr float kBelow = 1.0f - 0x1p-21f, kAbove = 1.0f + 0x1p-21f;
__device__ __forceinline__ uint32_t quant4_at(float4 v, float r) {
    return cvt_e4m3x2(v.x * r, v.y * r) | (cvt_e4m3x2(v.z * r, v.w * r) << 16);
}
// s at least 2^-100: below, 1 / s or the exact remainder may underflow.
__device__ __forceinline__ uint32_t quant4_normal(float4 v, float s, float inv) {
    const uint32_t lo = quant4_at(v, inv * kBelow), hi = quant4_at(v, inv * kAbove);
    if (lo == hi) return lo;
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t l = (lo >> (8 * i)) & 0xffu, h = (hi >> (8 * i)) & 0xffu;
        out |= (l == h ? l : quant1_decide(f[i], s, l, h)) << (8 * i);
    }
    return out;
}

__device__ __forceinline__ uint32_t quant4(float4 v, float s, float inv) {
    return s < 0x1p-100f ? quant4_wide(v, s) : quant4_normal(v, s, inv);
}

// The largest magnitude of four values, as the integer whose order it follows.
__device__ __forceinline__ uint32_t abs_bits(float4 v) {
    return max(max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu),
               max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
}

// The block of 128 values that a warp holds, 4 per lane (0 past the row's end): the packed bytes
// of the lane's values; *s receives the scale.  Returns the bytes; *finite is false (and bytes and
// scale 0) when a value was not finite.
__device__ __forceinline__ uint32_t quant_block(float4 v, float *s, bool *finite) {
    const uint32_t amax = __reduce_max_sync(0xffffffffu, abs_bits(v));
    const float sc = scale_of(amax);
    *s = sc;
    *finite = amax < 0x7f800000u;
    return sc > 0.0f ? quant4(v, sc, __frcp_rn(sc)) : 0u;
}

// silu(g) * u in fp32, a few ulp off: g / (1 + exp(-g)) with CUDA's expf and its division of 2 ulp (an
// IEEE division, whose slow path the unused rows of a tile take, made 64 tokens 410 us instead of
// 315).  From -80 on down, where exp(-g) leaves that division's range and then fp32's, the 1 is less
// than an ulp, and g exp(g) is the same.
constexpr float kSiluFar = -80.0f;
__device__ __forceinline__ float swiglu_near(float g, float u) {
    return __fdividef(g, 1.0f + expf(-g)) * u;
}
__device__ __forceinline__ float swiglu(float g, float u) {
    const bool far = g < kSiluFar;
    const float e = expf(far ? g : -g);
    return (far ? g * e : __fdividef(g, 1.0f + e)) * u;
}

// ------------------------------------------------------------------ launchers

// Launch behind the previous kernel of the stream (programmatic dependent launch): the kernel may
// start once every CTA of that one has called launch_dependents or ended, and sees its results
// after grid_dependency_wait.
template <typename... P, typename... Q>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                          cudaStream_t st, Q... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (err != cudaSuccess) return err;
    note_launches(1);
    return cudaGetLastError();
}

// ws: moe_route_workspace_size bytes.
cudaError_t launch_route_scored(const float *logits, int T, int E, int k,
                                const moe_route_rule &rule, int32_t *ids, float *w,
                                int32_t *counts, int32_t *offsets, int32_t *perm,
                                int32_t *inv_perm, uint32_t *status, void *ws, cudaStream_t st);

cudaError_t launch_scaled_quantize(const void *x, int dt, int T, int K, int64_t ldx, uint8_t *q,
                                   int64_t ldq, float *s, int64_t lds, uint32_t *status,
                                   cudaStream_t st);

struct ScaledMatmulArgs {
    const uint8_t *a;
    int64_t lda;
    const float *as;
    int64_t ldas;
    int M, K;
    const uint8_t *b;
    int64_t ldb;
    const float *bs;
    int N;
    void *out;
    int dt;
    int64_t ldo;
    uint32_t *status;
    uint64_t wait_ns;              // limit of every wait inside the tensor-core kernels
};
// The product on the kernel that suits its sizes, and the workspace it needs.
size_t scaled_matmul_ws_bytes(int M, int N, int K);
cudaError_t launch_scaled_matmul(const ScaledMatmulArgs &a, void *ws, cudaStream_t st);
// k_scaled_small.cu: M <= kSmallT.
cudaError_t launch_scaled_small(const ScaledMatmulArgs &a, cudaStream_t st);

constexpr int kScaledMaxDim = 1 << 16;             // hidden and ffn of scaled experts
constexpr int64_t kScaledMaxSlots = 1 << 24;       // (token, expert) pairs, the shared one's too

struct ScaledExpertsArgs {
    moe_scaled_weights w;
    const void *x;
    int x_dt;
    int T, k;
    const int32_t *ids;
    const float *rw;               // routing weights [T][k]
    const int32_t *offsets, *inv_perm;
    const float *gate;             // [T] or null
    void *out;
    int out_dt;
    uint32_t *status;
    uint64_t wait_ns;              // as of ScaledMatmulArgs
    float *h;                      // one token: h of every slot [slots][ffn]
};
// x quantised into the slots of its tokens: q [slots][hidden], scales [blocks][slots]; and the
// experts' runs of at most kScaledRun slots, with their number.
constexpr int kScaledRun = 128;
struct SliceArgs {
    const int32_t *offsets;
    int E, T, k, shared;
    Job *slices;
    int32_t *nslices;
};
cudaError_t launch_scaled_spread(const ScaledExpertsArgs &e, uint8_t *q, float *s, Job *slices,
                                 int32_t *nslices, cudaStream_t st);
// The layer on the kernels that suit T, and the workspace they need for exactly T tokens.
size_t scaled_experts_ws_bytes(const moe_scaled_weights &w, int T, int k);
cudaError_t launch_scaled_experts(const ScaledExpertsArgs &a, void *ws, cudaStream_t st);
// k_scaled_small.cu: T <= kSmallExpertsT, and the workspace for it.
size_t scaled_small_ws_bytes(int T, int k, int shared, int H, int F);
cudaError_t launch_scaled_experts_small(const ScaledExpertsArgs &a, void *ws, cudaStream_t st);

}  // namespace moe
