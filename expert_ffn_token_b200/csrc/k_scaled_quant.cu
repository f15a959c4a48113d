// k_scaled_quant.cu -- activations to e4m3 with one fp32 scale per row and 128 columns.
//
// Reads every value once and writes a byte per value and 4 bytes per 128: bound by memory.  A
// warp takes four rows of one column block, so that four loads are in flight per lane and the
// four scales, neighbours in the block-major scale array, go out together.
#include "scaled.cuh"

namespace moe {

namespace {

constexpr int kRows = 4;       // rows per warp

template <typename T, bool kVec>
__global__ void __launch_bounds__(256)
    k_scaled_quantize(const T *__restrict__ x, int rows, int K, int64_t ldx, uint8_t *__restrict__ q,
                      int64_t ldq, float *__restrict__ s, int64_t lds, uint32_t *status) {
    const int lane = threadIdx.x & 31;
    const int nb = sblocks(K);
    const int64_t unit = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    const int64_t rt = unit / nb;
    const int b = (int)(unit - rt * nb);
    const int64_t t0 = rt * kRows;
    if (t0 >= rows) return;
    const int c = b * kSBlk + lane * 4;
    float4 v[kRows];
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
    float mine = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        float sc;
        bool fin;
        const uint32_t p = quant_block(v[i], &sc, &fin);
        if (lane == i) mine = sc;
        bad = bad || !fin;
        if (t0 + i >= rows) continue;
        uint8_t *o = q + (t0 + i) * ldq + c;
        if (c + 3 < K) {
            *reinterpret_cast<uint32_t *>(o) = p;
        } else {
            for (int j = 0; j < 3; j++)
                if (c + j < K) o[j] = (uint8_t)(p >> (8 * j));
        }
    }
    if (lane < kRows && t0 + lane < rows) s[b * lds + t0 + lane] = mine;
    if (bad && lane == 0) set_status(status, MOE_ERR_NONFINITE);
}

}  // namespace

cudaError_t launch_scaled_quantize(const void *x, int dt, int T, int K, int64_t ldx, uint8_t *q,
                                   int64_t ldq, float *s, int64_t lds, uint32_t *status,
                                   cudaStream_t st) {
    if (T <= 0) return cudaSuccess;
    const int64_t units = (int64_t)((T + kRows - 1) / kRows) * sblocks(K);
    const unsigned grid = (unsigned)((units + 7) / 8);
    return with_dtype(dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        const E *p = static_cast<const E *>(x);
        // vector loads where every lane's four elements start on their natural boundary
        const bool vec = ((uintptr_t)x % (4 * sizeof(E))) == 0 && ldx % 4 == 0 && K % 4 == 0;
        if (vec)
            k_scaled_quantize<E, true><<<grid, 256, 0, st>>>(p, T, K, ldx, q, ldq, s, lds, status);
        else
            k_scaled_quantize<E, false><<<grid, 256, 0, st>>>(p, T, K, ldx, q, ldq, s, lds, status);
        note_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace moe
