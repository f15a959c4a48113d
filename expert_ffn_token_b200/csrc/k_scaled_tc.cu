// k_scaled_tc.cu -- products of scaled (e4m3, 128-block) operands on the 5th-generation tensor
// cores: the dense product and the experts' gate/up and down, for more tokens than the
// small-batch kernels take.
//
//   out[m][n] = sum_b as[b][m] bs[n/128][b] * P_b,   P_b = sum over the block's 128 k of a w
//
// P_b is one accumulator in tensor memory (four tcgen05.mma.kind::f8f6f4 of K = 32, exact
// products, fp32 sums); every block starts a new one.  The epilogue warps take it out of tensor
// memory and add P_b * (as * bs) to running totals in registers.
//
// Tile: 128 tokens (the MMA's N side, the tile's own count rounded up to 16) by two M = 128
// operands of weight rows: 256 rows of one matrix, or 128 gate rows and the 128 up rows of the
// same ffn values.  Weights sit on the M side so that an expert with few tokens wastes few MMA
// columns, and so that a tensor-memory lane is a weight row: the block scale of the weights is
// one number per operand and lanes write neighbouring outputs.  One persistent CTA per SM.
//
// Roles (384 threads; registers move from the first four warps to the epilogue):
//   warp 0        TMA producer: weight boxes of 128 rows x 128 bytes, token rows as boxes of 16
//                 or, for routed tokens, gathered four at a time
//   warp 1        tensor-memory allocation and the MMA issuer
//   warps 2-3     scales: as * bs of every column and block, into a ring
//   warps 4-11    epilogue: lane quarter (warp % 4), 64 columns each, both operands
// Every hand-off is an mbarrier and every wait is bounded (MOE_ERR_TIMEOUT in the status word).
#include <algorithm>

#include "scaled.cuh"
#include "tc_pipe.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int kNT = 128;                       // most tokens of a tile
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kOperand = 128 * kSBlk;     // bytes of 128 rows of one block
constexpr uint32_t kStage = 3 * kOperand;      // two weight operands and the tokens
constexpr int kStages = 4;
constexpr int kScales = 8;                     // depth of the scale ring
constexpr int kAccs = 2;                       // accumulator buffers of 2 x 128 columns
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;    // limit of every wait
// Registers: 384 threads launch with 168 each (64512); the first warpgroup keeps 64 and the two
// epilogue warpgroups take 216: 128 * 64 + 256 * 216 = 63488.
constexpr int kLaunchRegs = 168, kRoleRegs = 64, kEpiRegs = 216;
static_assert(128 * kRoleRegs + 256 * kEpiRegs <= kThreads * kLaunchRegs, "register split");

enum Mode { kGateUp, kDown, kDense };

struct TcArgs {
    int nkb;                     // blocks of k
    int rows;                    // weight rows per expert (gate/up: of each of the two)
    int row_tiles;
    int M;                       // dense: rows of a
    const Job *jobs;             // experts: written by k_scaled_jobs
    const int32_t *njobs;
    const int32_t *perm;
    int T, k, routed;            // routed = T * k
    const float *as;
    int64_t ldas;
    const float *ws0, *ws1;      // weight scales [expert][row blocks][nkb]; ws1: up
    int64_t ws_expert;
    uint8_t *hq;                 // gate/up: [slots][rows] and scales [row blocks][slots]
    float *hs;
    int64_t slots;
    void *out;
    int64_t ldo;
    uint32_t *status;
};

struct Tile {
    int e, rt, slot, n, npad;
    bool shared;
};

struct Walk {
    int j = 0, base = 0;
};

// Tile i (increasing) of the order: job, 128-token slice, row tile.
template <int kMode>
__device__ __forceinline__ bool tile_at(const TcArgs &a, int nj, Walk &c, int i, Tile &t) {
    while (c.j < nj) {
        const Job jb = kMode == kDense ? Job{0, 0, a.M, 0} : a.jobs[c.j];
        const int cnt = (jb.n + kNT - 1) / kNT * a.row_tiles;
        if (i < c.base + cnt) {
            const int sl = (i - c.base) / a.row_tiles;
            t.rt = (i - c.base) - sl * a.row_tiles;
            t.e = jb.expert;
            t.slot = jb.slot0 + sl * kNT;
            t.n = min(kNT, jb.n - sl * kNT);
            t.npad = (t.n + 15) & ~15;
            t.shared = jb.shared != 0;
            return true;
        }
        c.base += cnt;
        c.j++;
    }
    return false;
}

// silu(g) * u in fp32 with CUDA's expf and an IEEE division.
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fdiv_rn(g, 1.0f + expf(-g)) * u;
}

// The row of x that slot s of a tile reads.
__device__ __forceinline__ int token_of(const TcArgs &a, const Tile &t, int s) {
    if (t.shared) return s - a.routed;
    const int p = a.perm[s];
    if (p < 0 || p >= a.routed) {
        set_status(a.status, MOE_ERR_BOUNDS);
        return 0;
    }
    return p / a.k;
}

struct Shared {
    uint64_t full[kStages], empty[kStages], acc_full[kAccs], acc_empty[kAccs], sc_full[kScales],
        sc_empty[kScales], done;
    uint32_t tmem;
    int abort;
    alignas(16) float scale[kScales][2][kNT];
    alignas(16) uint32_t amax[2][kNT][4];        // gate/up: per column and lane quarter, by tile parity
};

constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + sizeof(Shared);
static_assert(kSmem <= 232448, "shared memory");

struct Pos {                          // ring position
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int d) {
        if (++s == d) {
            s = 0;
            ph ^= 1u;
        }
    }
};

__device__ __forceinline__ bool wait_slow(uint64_t *bar, uint32_t parity, int *abort,
                                       uint32_t *status) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (*(volatile int *)abort) return false;
        if (globaltimer() - t0 > kWaitNs) {
            *(volatile int *)abort = 1;
            set_status(status, MOE_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait1(Shared &S, uint64_t *bar, uint32_t parity, uint32_t *st) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, &S.abort, st);
}
// The same for a whole warp, with one answer.
__device__ __forceinline__ bool waitw(Shared &S, uint64_t *bar, uint32_t parity, uint32_t *st) {
    return __all_sync(0xffffffffu, wait1(S, bar, parity, st));
}

template <int kMode>
__device__ void produce(const TcArgs &a, Shared &S, uint8_t *ring, int nj, const CUtensorMap *w0,
                        const CUtensorMap *w1, const CUtensorMap *x) {
    const int lane = threadIdx.x & 31;
    Walk c;
    Tile t;
    Pos p;
    int issued = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && tile_at<kMode>(a, nj, c, i, t); i += gridDim.x) {
        int y[4];
        if (kMode == kGateUp) {
#pragma unroll
            for (int j = 0; j < 4; j++) y[j] = token_of(a, t, t.slot + min(4 * lane + j, t.n - 1));
        }
        for (int b = 0; b < a.nkb; b++) {
            if (!waitw(S, &S.empty[p.s], p.ph ^ 1u, a.status)) {
                ok = false;
                break;
            }
            uint8_t *st = ring + (size_t)p.s * kStage;
            uint64_t *bar = &S.full[p.s];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, 2 * kOperand + (uint32_t)t.npad * kSBlk);
                const int r0 = kMode == kGateUp ? t.rt * 128 : t.rt * 256;
                tma_load_3d(st, w0, b * kSBlk, r0, t.e, bar);
                tma_load_3d(st + kOperand, w1, b * kSBlk, kMode == kGateUp ? r0 : r0 + 128, t.e,
                            bar);
            }
            __syncwarp();
            uint8_t *xs = st + 2 * kOperand;
            if (kMode == kGateUp) {
                if (4 * lane < t.npad)
                    tma_gather4(xs + lane * 4 * kSBlk, x, b * kSBlk, y[0], y[1], y[2], y[3], bar);
            } else if (16 * lane < t.npad) {
                tma_load_2d(xs + lane * 16 * kSBlk, x, b * kSBlk, t.slot + 16 * lane, bar);
            }
            issued++;
            p.next(kStages);
        }
    }
    // leaving early: the copies in flight land before the CTA goes
    if (!ok) {
        for (int i = max(0, issued - kStages); i < issued; i++)
            mbar_wait_bounded(&S.full[i % kStages], (uint32_t)(i / kStages) & 1u, kWaitNs);
    }
}

template <int kMode>
__device__ void multiply(const TcArgs &a, Shared &S, uint8_t *ring, int nj, uint32_t tmem) {
    Walk c;
    Tile t;
    Pos p, q;
    for (int i = blockIdx.x; tile_at<kMode>(a, nj, c, i, t); i += gridDim.x) {
        const uint32_t idesc = instr_desc(0, 128, t.npad);
        for (int b = 0; b < a.nkb; b++) {
            if (!wait1(S, &S.acc_empty[q.s], q.ph ^ 1u, a.status) ||
                !wait1(S, &S.full[p.s], p.ph, a.status)) {
                umma_commit(&S.done);
                mbar_wait_bounded(&S.done, 0, kWaitNs);
                return;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(ring + (size_t)p.s * kStage);
            const uint32_t d = tmem + (uint32_t)q.s * 256u;
            const uint64_t x = smem_desc(st + 2 * kOperand, 1024, 2);
            const uint64_t w0 = smem_desc(st, 1024, 2), w1 = smem_desc(st + kOperand, 1024, 2);
#pragma unroll
            for (int j = 0; j < 4; j++) {    // 32 bytes of k a step: 2 units of 16 bytes
                umma_f8(d, w0 + 2 * j, x + 2 * j, idesc, j > 0);
                umma_f8(d + 128, w1 + 2 * j, x + 2 * j, idesc, j > 0);
            }
            umma_commit(&S.empty[p.s]);
            umma_commit(&S.acc_full[q.s]);
            p.next(kStages);
            q.next(kAccs);
        }
    }
}

template <int kMode>
__device__ void scales(const TcArgs &a, Shared &S, int nj, int half) {
    constexpr int kAhead = 4;           // blocks whose loads are issued together
    const int lane = threadIdx.x & 31;
    const int rb = (a.rows + kSBlk - 1) / kSBlk;
    Walk c;
    Tile t;
    Pos p;
    for (int i = blockIdx.x; tile_at<kMode>(a, nj, c, i, t); i += gridDim.x) {
        const float *as[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int col = half * 64 + j * 32 + lane;
            as[j] = col >= t.n ? nullptr
                    : a.as + (kMode == kGateUp ? token_of(a, t, t.slot + col) : t.slot + col);
        }
        const float *s0 = a.ws0 + t.e * a.ws_expert, *s1;
        if (kMode == kGateUp) {
            s0 += (int64_t)t.rt * a.nkb;
            s1 = a.ws1 + t.e * a.ws_expert + (int64_t)t.rt * a.nkb;
        } else {
            s0 += (int64_t)(2 * t.rt) * a.nkb;
            s1 = 2 * t.rt + 1 < rb ? s0 + a.nkb : s0;      // past the last rows: not stored
        }
        for (int b0 = 0; b0 < a.nkb; b0 += kAhead) {
            float v[kAhead][2], w[kAhead][2];
#pragma unroll
            for (int u = 0; u < kAhead; u++) {
                const int b = b0 + u;
                const bool in = b < a.nkb;
                v[u][0] = in && as[0] ? __ldg(as[0] + b * a.ldas) : 0.f;
                v[u][1] = in && as[1] ? __ldg(as[1] + b * a.ldas) : 0.f;
                w[u][0] = in ? __ldg(s0 + b) : 0.f;
                w[u][1] = in ? __ldg(s1 + b) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kAhead; u++) {
                if (b0 + u >= a.nkb) break;
                if (!waitw(S, &S.sc_empty[p.s], p.ph ^ 1u, a.status)) return;
                const int col = half * 64 + lane;
                S.scale[p.s][0][col] = v[u][0] * w[u][0];
                S.scale[p.s][0][col + 32] = v[u][1] * w[u][0];
                S.scale[p.s][1][col] = v[u][0] * w[u][1];
                S.scale[p.s][1][col + 32] = v[u][1] * w[u][1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.sc_full[p.s]);
                p.next(kScales);
            }
        }
    }
}

// Running totals of two columns in one 64-bit register pair.
__device__ __forceinline__ float2 pair(uint64_t v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    return (uint64_t)lo | ((uint64_t)hi << 32);
}
// acc += r * s for 16 columns, two at a time.
__device__ __forceinline__ void promote16(uint64_t *acc, const uint32_t (&r)[16], const float *s) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(s + i);
        asm("fma.rn.f32x2 %0, %1, %2, %0;"
            : "+l"(acc[i / 2]) : "l"(pair(r[i], r[i + 1])), "l"(v.x));
        asm("fma.rn.f32x2 %0, %1, %2, %0;"
            : "+l"(acc[i / 2 + 1]) : "l"(pair(r[i + 2], r[i + 3])), "l"(v.y));
    }
}

template <int kMode, typename T>
__device__ void finish(const TcArgs &a, Shared &S, int nj, uint32_t tmem) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const int c0 = half * 64;
    const uint32_t base = tmem + ((uint32_t)quad << 21) + (uint32_t)c0;   // lane quad * 32
    Walk c;
    Tile t;
    Pos q, p;
    uint32_t par = 0;
    for (int i = blockIdx.x; tile_at<kMode>(a, nj, c, i, t); i += gridDim.x) {
        uint64_t acc[2][32];            // two columns each
#pragma unroll
        for (int j = 0; j < 32; j++) acc[0][j] = acc[1][j] = 0u;
        const bool busy = c0 < t.npad;
        for (int b = 0; b < a.nkb; b++) {
            if (!waitw(S, &S.sc_full[p.s], p.ph, a.status)) return;
            if (!waitw(S, &S.acc_full[q.s], q.ph, a.status)) return;
            if (busy) {
                tc_fence_after();
                const uint32_t d = base + (uint32_t)q.s * 256u;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t r0[16], r1[16];
                    tmem_ld16(d + 16 * j, r0);
                    tmem_ld16(d + 128 + 16 * j, r1);
                    tmem_ld_wait(r0);
                    reg_tie(r1);
                    promote16(acc[0] + 8 * j, r0, S.scale[p.s][0] + c0 + 16 * j);
                    promote16(acc[1] + 8 * j, r1, S.scale[p.s][1] + c0 + 16 * j);
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&S.acc_empty[q.s]);
                mbar_arrive(&S.sc_empty[p.s]);
            }
            q.next(kAccs);
            p.next(kScales);
        }
        if (kMode == kGateUp) {
            // h, and its e4m3 form per token and 128 ffn values: the 128 lanes of the operand
            const int f = t.rt * 128 + quad * 32 + lane;
            uint32_t keep[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 32; j++) {
                const float2 g = pair(acc[0][j]), u = pair(acc[1][j]);
                const float h0 = silu_mul(g.x, u.x), h1 = silu_mul(g.y, u.y);
                acc[0][j] = pair(__float_as_uint(h0), __float_as_uint(h1));
                const uint32_t m0 =
                    __reduce_max_sync(0xffffffffu, __float_as_uint(h0) & 0x7fffffffu);
                const uint32_t m1 =
                    __reduce_max_sync(0xffffffffu, __float_as_uint(h1) & 0x7fffffffu);
                if (lane == ((2 * j) & 31)) keep[j >> 4] = m0;
                if (lane == ((2 * j + 1) & 31)) keep[j >> 4] = m1;
            }
            S.amax[par][c0 + lane][quad] = keep[0];
            S.amax[par][c0 + 32 + lane][quad] = keep[1];
            named_barrier(1 + half, 128);
            uint8_t *hq = a.hq + ((int64_t)t.slot + c0) * a.rows + f;
            float *hs = a.hs + t.rt * a.slots + t.slot + c0;
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
                if (c0 + j < t.n) {
                    float sc[2], inv[2];
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint4 m = *reinterpret_cast<const uint4 *>(S.amax[par][c0 + j + u]);
                        const uint32_t mx = max(max(m.x, m.y), max(m.z, m.w));
                        const bool fin = mx < 0x7f800000u;
                        sc[u] = fin ? __fdiv_rn(__uint_as_float(mx), kE4M3Max) : 0.f;
                        inv[u] = sc[u] > 0.f ? __frcp_rn(sc[u]) : 0.f;
                        if (!fin && c0 + j + u < t.n && quad == 0 && lane == 0)
                            set_status(a.status, MOE_ERR_NONFINITE);
                    }
                    const float2 h = pair(acc[0][j / 2]);
                    const uint32_t v = cvt_e4m3x2(sc[0] > 0.f ? h.x * inv[0] : 0.f,
                                                  sc[1] > 0.f ? h.y * inv[1] : 0.f);
                    const bool two = c0 + j + 1 < t.n;
                    if (f < a.rows) {
                        hq[0] = (uint8_t)v;
                        if (two) hq[a.rows] = (uint8_t)(v >> 8);
                    }
                    if (quad == 0 && lane == 0) {
                        hs[j] = sc[0];
                        if (two) hs[j + 1] = sc[1];
                    }
                }
                hq += 2 * (int64_t)a.rows;
            }
            par ^= 1u;
        } else {
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int r = t.rt * 256 + u * 128 + quad * 32 + lane;
                T *out = static_cast<T *>(a.out) + ((int64_t)t.slot + c0) * a.ldo + r;
                if (r < a.rows) {
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        const float2 v = pair(acc[u][j]);
                        if (c0 + 2 * j < t.n) out[0] = from_f32<T>(v.x);
                        if (c0 + 2 * j + 1 < t.n) out[a.ldo] = from_f32<T>(v.y);
                        out += 2 * a.ldo;
                    }
                }
            }
        }
    }
}

template <int kMode, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    k_scaled_tc(const TcArgs a, const __grid_constant__ CUtensorMap w0,
                const __grid_constant__ CUtensorMap w1, const __grid_constant__ CUtensorMap x) {
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~uintptr_t(1023));
    Shared &S = *reinterpret_cast<Shared *>(ring + (size_t)kStages * kStage);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; i++) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < kAccs; i++) {
            mbar_init(&S.acc_full[i], 1);
            mbar_init(&S.acc_empty[i], kEpiWarps);
        }
        for (int i = 0; i < kScales; i++) {
            mbar_init(&S.sc_full[i], 2);
            mbar_init(&S.sc_empty[i], kEpiWarps);
        }
        mbar_init(&S.done, 1);
        S.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&S.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int nj = kMode == kDense ? 1 : *a.njobs;
    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
        if (warp == 0)
            produce<kMode>(a, S, ring, nj, &w0, &w1, &x);
        else if (warp == 1) {
            if ((threadIdx.x & 31) == 0) multiply<kMode>(a, S, ring, nj, tmem);
        } else
            scales<kMode>(a, S, nj, warp - 2);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        finish<kMode, T>(a, S, nj, tmem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The experts' job list: one job per expert with tokens, the shared one last.  One CTA.
__global__ void __launch_bounds__(1024)
    k_scaled_jobs(const int32_t *__restrict__ offsets, int E, int T, int k, int shared, Job *jobs,
                  int32_t *njobs, uint32_t *status) {
    __shared__ int s_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, A = T * k;
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 1024) {
        const int e = e0 + threadIdx.x;
        int n = 0, o = 0;
        if (e < E) {
            o = offsets[e];
            const int o1 = offsets[e + 1];
            n = o1 - o;
            if (o < 0 || o1 > A || n < 0) {      // not what a router wrote
                set_status(status, MOE_ERR_BOUNDS);
                n = 0;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, n > 0);
        if (lane == 0) s_warp[warp] = __popc(m);
        __syncthreads();
        int at = base, all = 0;
        for (int w = 0; w < 32; w++) {
            at += w < warp ? s_warp[w] : 0;
            all += s_warp[w];
        }
        if (n > 0) jobs[at + __popc(m & ((1u << lane) - 1u))] = Job{e, o, n, 0};
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        if (shared) jobs[base] = Job{E, A, T, 1};
        *njobs = base + (shared ? 1 : 0);
    }
}

// out[t] = sum_j w[t][j] y[slot of (t, j)] (+ gate[t] y[routed + t]): one CTA per token.
template <typename T>
__global__ void __launch_bounds__(256)
    k_scaled_combine(const float *__restrict__ y, const int32_t *__restrict__ inv_perm,
                     const int32_t *__restrict__ ids, const float *__restrict__ w,
                     const float *__restrict__ gate, int tokens, int k, int E, int shared, int H,
                     T *__restrict__ out, uint32_t *status) {
    __shared__ int s_slot[kMaxK + 1];
    __shared__ float s_w[kMaxK + 1];
    const int t = blockIdx.x, A = tokens * k;
    if ((int)threadIdx.x < k) {
        const int s = inv_perm[t * k + threadIdx.x], e = ids[t * k + threadIdx.x];
        const bool in = s >= 0 && s < A && e >= 0 && e < E;
        if (!in) set_status(status, MOE_ERR_BOUNDS);
        s_slot[threadIdx.x] = in ? s : -1;
        s_w[threadIdx.x] = w[t * k + threadIdx.x];
    }
    if (threadIdx.x == 0) {
        s_slot[k] = shared ? A + t : -1;
        s_w[k] = shared ? (gate ? gate[t] : 1.0f) : 0.f;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < H / 4; c += blockDim.x) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j <= k; j++) {
            if (s_slot[j] < 0) continue;
            const float4 v = __ldg(reinterpret_cast<const float4 *>(y + (int64_t)s_slot[j] * H) + c);
            const float f = s_w[j];
            s.x = fmaf(f, v.x, s.x);
            s.y = fmaf(f, v.y, s.y);
            s.z = fmaf(f, v.z, s.z);
            s.w = fmaf(f, v.w, s.w);
        }
        T *o = out + (int64_t)t * H + 4 * c;
        o[0] = from_f32<T>(s.x);
        o[1] = from_f32<T>(s.y);
        o[2] = from_f32<T>(s.z);
        o[3] = from_f32<T>(s.w);
    }
}

// ---------------------------------------------------------------- host side

// A map of 8-bit rows, 128-byte swizzle: [outer][rows][cols], boxes of 128 bytes x box_rows.
bool encode(CUtensorMap *m, const void *base, int cols, int64_t rows, int64_t stride, int outer,
            int box_rows) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)(stride * rows)};
    const cuuint32_t box[3] = {kSBlk, (cuuint32_t)box_rows, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, outer > 0 ? 3 : 2, const_cast<void *>(base), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kMode, typename T>
cudaError_t run_tc(const TcArgs &a, const CUtensorMap &w0, const CUtensorMap &w1,
                   const CUtensorMap &x, int64_t most_tiles, cudaStream_t st) {
    auto kernel = k_scaled_tc<kMode, T>;
    // the register split needs every register of the launch it was made for
    static const bool fits = [&] {
        cudaFuncAttributes at{};
        return cudaFuncGetAttributes(&at, kernel) == cudaSuccess && at.numRegs >= kLaunchRegs;
    }();
    if (!fits) return cudaErrorLaunchOutOfResources;
    cudaError_t err = ensure_smem(kernel, kSmem);
    if (err != cudaSuccess) return err;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    kernel<<<(unsigned)std::min<int64_t>(sms, most_tiles), kThreads, kSmem, st>>>(a, w0, w1, x);
    note_launches(1);
    return cudaGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct ExpertsWs {
    size_t xq, xs, hq, hs, y, jobs, njobs, total;
    int64_t slots;
};

ExpertsWs experts_ws(const moe_scaled_weights &w, int T, int k) {
    ExpertsWs L{};
    size_t p = 0;
    auto take = [&](size_t bytes) {
        const size_t o = p;
        p = align256(p + bytes);
        return o;
    };
    L.slots = (int64_t)T * k + (w.shared ? T : 0);
    L.xq = take((size_t)T * w.hidden);
    L.xs = take((size_t)sblocks(w.hidden) * T * 4);
    L.hq = take((size_t)L.slots * w.ffn);
    L.hs = take((size_t)sblocks(w.ffn) * L.slots * 4);
    L.y = take((size_t)L.slots * w.hidden * 4);
    L.jobs = take(sizeof(Job) * ((size_t)std::min<int64_t>(w.n_experts, (int64_t)T * k) + 1));
    L.njobs = take(4);
    L.total = p;
    return L;
}

cudaError_t experts_tc(const ScaledExpertsArgs &e, uint8_t *ws, cudaStream_t st) {
    const moe_scaled_weights &w = e.w;
    const ExpertsWs L = experts_ws(w, e.T, e.k);
    const int n = w.n_experts + w.shared, H = w.hidden, F = w.ffn;
    Job *jobs = reinterpret_cast<Job *>(ws + L.jobs);
    int32_t *njobs = reinterpret_cast<int32_t *>(ws + L.njobs);
    float *xs = reinterpret_cast<float *>(ws + L.xs);
    CUtensorMap gate, up, down, x, h;
    if (!encode(&gate, w.d_gate, H, F, H, n, 128) || !encode(&up, w.d_up, H, F, H, n, 128) ||
        !encode(&down, w.d_down, F, H, F, n, 128) || !encode(&x, ws + L.xq, H, e.T, H, 0, 1) ||
        !encode(&h, ws + L.hq, F, L.slots, F, 0, 16))
        return cudaErrorInvalidValue;
    k_scaled_jobs<<<1, 1024, 0, st>>>(e.offsets, w.n_experts, e.T, e.k, w.shared, jobs, njobs,
                                      e.status);
    note_launches(1);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    err = launch_scaled_quantize(e.x, e.x_dt, e.T, H, H, ws + L.xq, H, xs, e.T, e.status, st);
    if (err != cudaSuccess) return err;
    // an upper bound on the 128-token slices of all jobs
    const int64_t slices = L.slots / kNT + std::min<int64_t>(w.n_experts, (int64_t)e.T * e.k) + 1;
    TcArgs a{};
    a.jobs = jobs;
    a.njobs = njobs;
    a.perm = e.perm;
    a.T = e.T;
    a.k = e.k;
    a.routed = e.T * e.k;
    a.status = e.status;
    a.slots = L.slots;
    a.hq = ws + L.hq;
    a.hs = reinterpret_cast<float *>(ws + L.hs);
    a.nkb = sblocks(H);
    a.rows = F;
    a.row_tiles = sblocks(F);
    a.as = xs;
    a.ldas = e.T;
    a.ws0 = w.d_gate_s;
    a.ws1 = w.d_up_s;
    a.ws_expert = (int64_t)sblocks(F) * sblocks(H);
    err = run_tc<kGateUp, float>(a, gate, up, x, slices * a.row_tiles, st);
    if (err != cudaSuccess) return err;
    a.nkb = sblocks(F);
    a.rows = H;
    a.row_tiles = (H + 255) / 256;
    a.as = a.hs;
    a.ldas = L.slots;
    a.ws0 = w.d_down_s;
    a.out = ws + L.y;
    a.ldo = H;
    err = run_tc<kDown, float>(a, down, down, h, slices * a.row_tiles, st);
    if (err != cudaSuccess) return err;
    return with_dtype(e.out_dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        k_scaled_combine<E><<<e.T, 256, 0, st>>>(reinterpret_cast<const float *>(ws + L.y),
                                                 e.inv_perm, e.ids, e.rw, e.gate, e.T, e.k,
                                                 w.n_experts, w.shared, H,
                                                 static_cast<E *>(e.out), e.status);
        note_launches(1);
        return cudaGetLastError();
    });
}

cudaError_t matmul_tc(const ScaledMatmulArgs &m, cudaStream_t st) {
    CUtensorMap b, x;
    if (!encode(&b, m.b, m.K, m.N, m.ldb, 1, 128) || !encode(&x, m.a, m.K, m.M, m.lda, 0, 16))
        return cudaErrorInvalidValue;
    TcArgs a{};
    a.nkb = sblocks(m.K);
    a.rows = m.N;
    a.row_tiles = (m.N + 255) / 256;
    a.M = m.M;
    a.as = m.as;
    a.ldas = m.ldas;
    a.ws0 = m.bs;
    a.out = m.out;
    a.ldo = m.ldo;
    a.status = m.status;
    const int64_t tiles = (int64_t)((m.M + kNT - 1) / kNT) * a.row_tiles;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    return with_dtype(m.dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        return run_tc<kDense, E>(a, b, b, x, tiles, st);
    });
}

}  // namespace

size_t scaled_matmul_ws_bytes(int, int, int) { return 0; }

cudaError_t launch_scaled_matmul(const ScaledMatmulArgs &a, void *, cudaStream_t st) {
    return a.M <= kSmallT ? launch_scaled_small(a, st) : matmul_tc(a, st);
}

size_t scaled_experts_ws_bytes(const moe_scaled_weights &w, int T, int k) {
    return T <= kSmallT ? align256(scaled_small_h_bytes(T, k, w.shared, w.ffn))
                        : experts_ws(w, T, k).total;
}

cudaError_t launch_scaled_experts(const ScaledExpertsArgs &a, void *ws, cudaStream_t st) {
    if (a.T > kSmallT) return experts_tc(a, static_cast<uint8_t *>(ws), st);
    ScaledExpertsArgs s = a;
    s.h = static_cast<float *>(ws);
    return launch_scaled_experts_small(s, st);
}

}  // namespace moe
