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
// Tile: 128 tokens (the MMA's M side) by 256 weight rows (N): rows of one matrix, or 128 gate rows
// and the 128 up rows of the same ffn values.  Tokens sit on the M side so that a tensor-memory
// lane is a token: an epilogue thread's scale is then one number per block and operand.  With the weights on the M side the scale changes from column to column and has to
// be read from shared memory, two 16-byte loads per four elements; the loads, not the
// additions, then bound the kernel (1380 clocks per block of 128 k against 512 of MMA).  An
// expert with few tokens leaves rows of the MMA unused, which costs nothing that counts: it is
// bound by its weights' bytes.  One persistent CTA per SM.
//
// Roles (384 threads; registers move from the first four warps to the epilogue):
//   warp 0        TMA producer: weight boxes of 128 rows x 128 bytes, token rows as boxes of 16
//                 or, for routed tokens, gathered four at a time
//   warp 1        tensor-memory allocation and the MMA issuer
//   warps 2-3     scales: as * bs of every token, block and operand, into a ring, loaded four
//                 blocks ahead
//   warps 4-11    epilogue: lane quarter (warp % 4), 64 columns of each 128-row operand
// Every hand-off is an mbarrier and every wait is bounded (MOE_ERR_TIMEOUT in the status word).
#include <algorithm>

#include "route_dev.cuh"
#include "scaled.cuh"
#include "tc_pipe.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int kMT = 128;                       // most tokens of a tile
constexpr int kNW = 256;                       // weight rows of a tile (gate/up: 128 + 128)
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kOperand = 128 * kSBlk;     // bytes of 128 rows of one block
constexpr uint32_t kStage = 3 * kOperand;      // the weights' two operands and the tokens
constexpr int kStages = 4;
constexpr int kAccs = 2;                       // accumulator buffers of 256 columns
constexpr int kScales = 8;                     // depth of the scale ring
constexpr int kAhead = 4;                      // blocks whose scales are loaded ahead
constexpr int kPatch = 16;                     // columns per turn through shared memory (stores)
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;    // limit of every wait
// Registers: 384 threads launch with 168 each (64512); the first warpgroup keeps 96 and the two
// epilogue warpgroups take 200: 128 * 96 + 256 * 200 = 63488.
constexpr int kLaunchRegs = 168, kRoleRegs = 96, kEpiRegs = 200;
static_assert(sizeof(Job) == sizeof(int4), "a slice is loaded as one vector");
static_assert(128 * kRoleRegs + 256 * kEpiRegs <= kThreads * kLaunchRegs, "register split");

enum Mode { kGateUp, kDown, kDense };

struct TcArgs {
    int nkb;                     // blocks of k
    int rows;                    // weight rows per expert (gate/up: of each of the two)
    int row_tiles;
    int M;                       // dense: rows of a
    const Job *slices;           // experts: runs of up to 128 slots (k_scaled_slices)
    const int32_t *nslices;
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
    bool vec;                    // out rows are 32-byte aligned and rows a multiple of 16
    uint32_t *status;
};

struct Tile {
    int e, rt, slot, n, npad;
    bool shared;
};

// Tile i: row tiles innermost, so that the CTAs that run at the same time share an expert's
// weights (its slices follow one another) and a slice's tokens.
template <int kMode>
__device__ __forceinline__ Tile tile_at(const TcArgs &a, int i) {
    Tile t;
    const int s = i / a.row_tiles;
    t.rt = i - s * a.row_tiles;
    if (kMode == kDense) {
        t.e = 0;
        t.slot = s * kMT;
        t.n = min(kMT, a.M - t.slot);
        t.shared = false;
    } else {
        const int4 v = __ldg(reinterpret_cast<const int4 *>(a.slices) + s);
        t.e = v.x;
        t.slot = v.y;
        t.n = v.z;
        t.shared = v.w != 0;
    }
    t.npad = (t.n + 15) & ~15;
    return t;
}

// silu(g) * u in fp32 with CUDA's expf and its approximate division (2 ulp; a denominator past
// 2^126 gives 0, where the quotient is below 2^-119).
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fdividef(g, 1.0f + expf(-g)) * u;
}

// The row of x that a slot reads is its entry of perm over k; the shared expert's slots follow
// the routed ones in token order.  The entry is loaded ahead of its use.
__device__ __forceinline__ int slot_entry(const TcArgs &a, const Tile &t, int s) {
    return t.shared ? (s - a.routed) * a.k : __ldg(a.perm + s);
}
__device__ __forceinline__ int entry_token(const TcArgs &a, int p) {
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
    float2 scale[kScales][kMT];
    uint32_t amax[2][2][kMT];             // gate/up: by tile parity and column half, per token
    float patch[kEpiWarps][32][kPatch + 1];
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
__device__ void produce(const TcArgs &a, Shared &S, uint8_t *ring, int tiles, const CUtensorMap *w0,
                        const CUtensorMap *w1, const CUtensorMap *x) {
    const int lane = threadIdx.x & 31;
    Pos p;
    int issued = 0;
    bool ok = true;
    int i = blockIdx.x;
    if (i >= tiles) return;
    Tile next = tile_at<kMode>(a, i);
    int entry[4] = {0, 0, 0, 0};
    auto entries = [&] {
        if (kMode == kGateUp) {
#pragma unroll
            for (int j = 0; j < 4; j++)
                entry[j] = slot_entry(a, next, next.slot + min(4 * lane + j, next.n - 1));
        }
    };
    entries();
    for (; ok && i < tiles; i += gridDim.x) {
        const Tile t = next;
        int y[4];
#pragma unroll
        for (int j = 0; j < 4; j++) y[j] = kMode == kGateUp ? entry_token(a, entry[j]) : 0;
        // the next tile's place and token rows arrive while this one's blocks are issued
        const bool more = i + gridDim.x < tiles;
        if (more) next = tile_at<kMode>(a, i + gridDim.x);
        for (int b = 0; b < a.nkb; b++) {
            if (!waitw(S, &S.empty[p.s], p.ph ^ 1u, a.status)) {
                ok = false;
                break;
            }
            uint8_t *st = ring + (size_t)p.s * kStage;
            uint64_t *bar = &S.full[p.s];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, 2 * kOperand + (uint32_t)t.npad * kSBlk);
                const int r0 = kMode == kGateUp ? t.rt * 128 : t.rt * kNW;
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
            if (b == 0 && more) entries();
        }
    }
    // leaving early: the copies in flight land before the CTA goes
    if (!ok) {
        for (int j = max(0, issued - kStages); j < issued; j++)
            mbar_wait_bounded(&S.full[j % kStages], (uint32_t)(j / kStages) & 1u, kWaitNs);
    }
}

__device__ void multiply(const TcArgs &a, Shared &S, uint8_t *ring, int tiles, uint32_t tmem) {
    Pos p, q;
    constexpr uint32_t idesc = instr_desc(0, kMT, kNW);
    for (int i = blockIdx.x; i < tiles; i += gridDim.x) {
        for (int b = 0; b < a.nkb; b++) {
            if (!wait1(S, &S.acc_empty[q.s], q.ph ^ 1u, a.status) ||
                !wait1(S, &S.full[p.s], p.ph, a.status)) {
                umma_commit(&S.done);
                mbar_wait_bounded(&S.done, 0, kWaitNs);
                return;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(ring + (size_t)p.s * kStage);
            const uint32_t d = tmem + (uint32_t)(q.s * kNW);
            const uint64_t x = smem_desc(st + 2 * kOperand, 1024, 2), w = smem_desc(st, 1024, 2);
#pragma unroll
            for (int j = 0; j < 4; j++)      // 32 bytes of k a step: 2 units of 16 bytes
                umma_f8(d, x + 2 * j, w + 2 * j, idesc, j > 0);
            umma_commit(&S.empty[p.s]);
            umma_commit(&S.acc_full[q.s]);
            p.next(kStages);
            q.next(kAccs);
        }
    }
}

// Warps 2 and 3: the scales of every tile and block, in the order the epilogue takes them: the
// token's scale times the two operands' weight scales, one pair per token.  Loads run kAhead
// blocks ahead of the ring's writes, across tiles.
template <int kMode>
struct ScaleStream {
    struct Set {
        float v[2], w0, w1;
    };
    int i, b, entry[2];
    Tile t, next;
    const float *as[2], *s0, *s1;

    __device__ __forceinline__ void look(const TcArgs &a, int row) {
        if (kMode == kGateUp) {
#pragma unroll
            for (int j = 0; j < 2; j++)
                entry[j] = slot_entry(a, next, next.slot + min(row + 32 * j, next.n - 1));
        }
    }
    __device__ __forceinline__ void open(const TcArgs &a, int row) {
        t = next;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int r = row + 32 * j;
            as[j] = r >= t.n ? nullptr
                    : a.as + (kMode == kGateUp ? entry_token(a, entry[j]) : t.slot + r);
        }
        s0 = a.ws0 + t.e * a.ws_expert;
        if (kMode == kGateUp) {
            s0 += (int64_t)t.rt * a.nkb;
            s1 = a.ws1 + t.e * a.ws_expert + (int64_t)t.rt * a.nkb;
        } else {
            s0 += (int64_t)(2 * t.rt) * a.nkb;
            s1 = t.rt * kNW + kSBlk < a.rows ? s0 + a.nkb : s0;    // past the last rows: not stored
        }
    }
    __device__ __forceinline__ void start(const TcArgs &a, int row) {
        i = blockIdx.x;
        b = 0;
        next = tile_at<kMode>(a, i);
        look(a, row);
        open(a, row);
    }
    __device__ __forceinline__ void load(const TcArgs &a, int tiles, int row, Set &c) {
        if (i >= tiles) return;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            c.v[j] = 0.f;
            if (as[j]) {
                c.v[j] = __ldg(as[j]);
                as[j] += a.ldas;
            }
        }
        c.w0 = __ldg(s0 + b);
        c.w1 = __ldg(s1 + b);
        const bool more = i + (int)gridDim.x < tiles;
        if (b == 0 && more) {
            next = tile_at<kMode>(a, i + gridDim.x);
            look(a, row);
        }
        if (++b == a.nkb) {
            b = 0;
            i += gridDim.x;
            if (more) open(a, row);
        }
    }
};

template <int kMode>
__device__ void scales(const TcArgs &a, Shared &S, int tiles, int which) {
    const int lane = threadIdx.x & 31, row = which * 64 + lane;
    if ((int)blockIdx.x >= tiles) return;
    ScaleStream<kMode> ss;
    typename ScaleStream<kMode>::Set c[kAhead];
    ss.start(a, row);
#pragma unroll
    for (int u = 0; u < kAhead; u++) ss.load(a, tiles, row, c[u]);
    const int mine = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int64_t total = (int64_t)mine * a.nkb;
    Pos p;
    for (int64_t b0 = 0; b0 < total; b0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (b0 + u >= total) break;
            if (!waitw(S, &S.sc_empty[p.s], p.ph ^ 1u, a.status)) return;
            S.scale[p.s][row] = make_float2(c[u].v[0] * c[u].w0, c[u].v[0] * c[u].w1);
            S.scale[p.s][row + 32] = make_float2(c[u].v[1] * c[u].w0, c[u].v[1] * c[u].w1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.sc_full[p.s]);
            p.next(kScales);
            ss.load(a, tiles, row, c[u]);
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
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    return pair(__float_as_uint(lo), __float_as_uint(hi));
}
// acc += r * s for 32 columns, two at a time.
__device__ __forceinline__ void promote32(uint64_t *acc, const uint32_t (&r)[32], uint64_t s) {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        asm("fma.rn.f32x2 %0, %1, %2, %0;"
            : "+l"(acc[i / 2]) : "l"(pair(r[i], r[i + 1])), "l"(s));
}

__device__ __forceinline__ void store32B(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, float *) { return 0u; }
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16 *) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half *) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 16 columns (8 pairs) of this lane's row at p, 32-byte aligned.
template <typename T>
__device__ __forceinline__ void store16(T *p, const uint64_t *acc) {
    uint32_t v[8];
    if (sizeof(T) == 4) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = (uint32_t)acc[4 * h + i];
                v[2 * i + 1] = (uint32_t)(acc[4 * h + i] >> 32);
            }
            store32B(p + 8 * h, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 f = pair(acc[i]);
            v[i] = pack2(f.x, f.y, (T *)nullptr);
        }
        store32B(p, v);
    }
}

template <int kMode, typename T>
__device__ void finish(const TcArgs &a, Shared &S, int tiles, uint32_t tmem) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t base = tmem + ((uint32_t)quad << 21) + (uint32_t)(half * 64);  // lane quad * 32
    Pos q, p;
    uint32_t par = 0;
    int i = blockIdx.x;
    if (i >= tiles) return;
    Tile next = tile_at<kMode>(a, i);
    for (; i < tiles; i += gridDim.x) {
        const Tile t = next;
        if (i + (int)gridDim.x < tiles) next = tile_at<kMode>(a, i + gridDim.x);
        uint64_t acc[2][32];            // two columns each
#pragma unroll
        for (int j = 0; j < 32; j++) acc[0][j] = acc[1][j] = 0u;
        const bool busy = quad * 32 < t.n;
        for (int b = 0; b < a.nkb; b++) {
            if (!waitw(S, &S.sc_full[p.s], p.ph, a.status)) return;
            const float2 f = S.scale[p.s][row];
            if (!waitw(S, &S.acc_full[q.s], q.ph, a.status)) return;
            if (busy) {
                tc_fence_after();
                const uint32_t d = base + (uint32_t)(q.s * kNW);
                const uint64_t s0 = pair(f.x, f.x), s1 = pair(f.y, f.y);
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    uint32_t r0[32], r1[32];
                    tmem_ld32(d + 32 * j, r0);
                    tmem_ld32(d + 128 + 32 * j, r1);
                    tmem_ld_wait(r0);
                    reg_tie(r1);
                    promote32(acc[0] + 16 * j, r0, s0);
                    promote32(acc[1] + 16 * j, r1, s1);
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
        if (!busy) continue;
        if (kMode == kGateUp) {
            // h, and its e4m3 form per token and 128 ffn values: this thread's 64 and the other
            // column half's
            uint32_t m = 0u;
#pragma unroll
            for (int j = 0; j < 32; j++) {
                const float2 g = pair(acc[0][j]), u = pair(acc[1][j]);
                const float h0 = silu_mul(g.x, u.x), h1 = silu_mul(g.y, u.y);
                acc[0][j] = pair(h0, h1);
                m = max(m, max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu));
            }
            S.amax[par][half][row] = m;
            named_barrier(1 + quad, 64);
            m = max(m, S.amax[par][half ^ 1][row]);
            par ^= 1u;
            if (row < t.n) {
                const bool fin = m < 0x7f800000u;
                const float sc = fin ? __fdiv_rn(__uint_as_float(m), kE4M3Max) : 0.f;
                // h / sc as (h * pre) * (1 / (sc * pre)): pre keeps the reciprocal of a tiny scale finite
                const float pre = sc < 0x1p-100f ? 0x1p100f : 1.0f;
                const float inv = sc > 0.f ? __frcp_rn(sc * pre) : 0.f;
                const int64_t slot = (int64_t)t.slot + row;
                if (half == 0) {
                    a.hs[t.rt * a.slots + slot] = sc;
                    if (!fin) set_status(a.status, MOE_ERR_NONFINITE);
                }
                const int f = t.rt * 128 + half * 64;
                uint8_t *hq = a.hq + slot * a.rows + f;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t v[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const float2 x = pair(acc[0][8 * j + 2 * u]);
                        const float2 y = pair(acc[0][8 * j + 2 * u + 1]);
                        v[u] = cvt_e4m3x2(x.x * pre * inv, x.y * pre * inv) |
                               (cvt_e4m3x2(y.x * pre * inv, y.y * pre * inv) << 16);
                        if (!fin) v[u] = 0u;
                    }
                    if (f + 16 * j < a.rows)
                        *reinterpret_cast<uint4 *>(hq + 16 * j) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        } else {
            T *out = static_cast<T *>(a.out) + ((int64_t)t.slot + row) * a.ldo;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int r0 = t.rt * kNW + u * 128 + half * 64;
                if (a.vec) {
                    // 32 bytes of a row per lane and store
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (row < t.n && r0 + 16 * j < a.rows)
                            store16(out + r0 + 16 * j, acc[u] + 8 * j);
                } else {
                    // rows of any alignment: 16 columns at a time through shared memory, so that
                    // a warp writes runs of a row
                    float (&P)[32][kPatch + 1] = S.patch[warp - kEpiWarp0];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
#pragma unroll
                        for (int x = 0; x < 8; x++) {
                            const float2 v = pair(acc[u][8 * j + x]);
                            P[lane][2 * x] = v.x;
                            P[lane][2 * x + 1] = v.y;
                        }
                        __syncwarp();
                        const int col = r0 + 16 * j + (lane & 15);
                        const int first = quad * 32 + (lane >> 4);
                        T *o = static_cast<T *>(a.out) + ((int64_t)t.slot + first) * a.ldo + col;
                        if (col < a.rows) {
                            for (int y = 0; y < 16 && first + 2 * y < t.n; y++, o += 2 * a.ldo)
                                *o = from_f32<T>(P[(lane >> 4) + 2 * y][lane & 15]);
                        }
                        __syncwarp();
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
    const int tiles = (kMode == kDense ? (a.M + kMT - 1) / kMT : *a.nslices) * a.row_tiles;
    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
        if (warp == 0)
            produce<kMode>(a, S, ring, tiles, &w0, &w1, &x);
        if (warp == 1) {
            if ((threadIdx.x & 31) == 0) multiply(a, S, ring, tiles, tmem);
        }
        if (warp >= 2) scales<kMode>(a, S, tiles, warp - 2);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        finish<kMode, T>(a, S, tiles, tmem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The runs of up to 128 slots of every expert with tokens, ascending, the shared one's last: the
// tiles' token side.  One CTA.
__global__ void __launch_bounds__(1024)
    k_scaled_slices(const int32_t *__restrict__ offsets, int E, int T, int k, int shared,
                    Job *slices, int32_t *nslices, uint32_t *status) {
    __shared__ int s_first[kMaxE];
    __shared__ int s_warp[33];
    const int A = T * k;
    for (int e = threadIdx.x; e < E; e += 1024) {
        const int o = offsets[e], o1 = offsets[e + 1];
        const bool fits = o >= 0 && o <= o1 && o1 <= A;      // else not what a router wrote
        if (!fits) set_status(status, MOE_ERR_BOUNDS);
        s_first[e] = fits ? (o1 - o + kMT - 1) / kMT : 0;
    }
    __syncthreads();
    // overlapping runs of damaged offsets could pass the list's end: those are left out too
    const int most = A / kMT + min(E, A);
    const int n = min(block_exclusive_scan<1024>(s_first, E, s_warp), most);
    for (int e = threadIdx.x; e < E; e += 1024) {
        const int o = offsets[e], o1 = offsets[e + 1];
        if (!(o >= 0 && o <= o1 && o1 <= A)) continue;
        for (int s = o, j = s_first[e]; s < o1 && j < most; s += kMT, j++)
            slices[j] = Job{e, s, min(kMT, o1 - s), 0};
    }
    const int ns = shared ? (T + kMT - 1) / kMT : 0;
    for (int j = threadIdx.x; j < ns; j += 1024)
        slices[n + j] = Job{E, A + j * kMT, min(kMT, T - j * kMT), 1};
    if (threadIdx.x == 0) *nslices = n + ns;
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
    size_t xq, xs, hq, hs, y, slices, nslices, total;
    int64_t slots, most_slices;
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
    L.most_slices = (int64_t)T * k / kMT + std::min<int64_t>(w.n_experts, (int64_t)T * k) +
                    (w.shared ? (T + kMT - 1) / kMT : 0);
    L.slices = take(sizeof(Job) * (size_t)L.most_slices);
    L.nslices = take(4);
    L.total = p;
    return L;
}

cudaError_t experts_tc(const ScaledExpertsArgs &e, uint8_t *ws, cudaStream_t st) {
    const moe_scaled_weights &w = e.w;
    const ExpertsWs L = experts_ws(w, e.T, e.k);
    const int n = w.n_experts + w.shared, H = w.hidden, F = w.ffn;
    Job *slices = reinterpret_cast<Job *>(ws + L.slices);
    int32_t *nslices = reinterpret_cast<int32_t *>(ws + L.nslices);
    float *xs = reinterpret_cast<float *>(ws + L.xs);
    CUtensorMap gate, up, down, x, h;
    if (!encode(&gate, w.d_gate, H, F, H, n, 128) || !encode(&up, w.d_up, H, F, H, n, 128) ||
        !encode(&down, w.d_down, F, H, F, n, 128) || !encode(&x, ws + L.xq, H, e.T, H, 0, 1) ||
        !encode(&h, ws + L.hq, F, L.slots, F, 0, 16))
        return cudaErrorInvalidValue;
    k_scaled_slices<<<1, 1024, 0, st>>>(e.offsets, w.n_experts, e.T, e.k, w.shared, slices,
                                        nslices, e.status);
    note_launches(1);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    err = launch_scaled_quantize(e.x, e.x_dt, e.T, H, H, ws + L.xq, H, xs, e.T, e.status, st);
    if (err != cudaSuccess) return err;
    TcArgs a{};
    a.slices = slices;
    a.nslices = nslices;
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
    err = run_tc<kGateUp, float>(a, gate, up, x, L.most_slices * a.row_tiles, st);
    if (err != cudaSuccess) return err;
    a.nkb = sblocks(F);
    a.rows = H;
    a.row_tiles = (H + kNW - 1) / kNW;
    a.as = a.hs;
    a.ldas = L.slots;
    a.ws0 = w.d_down_s;
    a.out = ws + L.y;
    a.ldo = H;
    a.vec = true;
    err = run_tc<kDown, float>(a, down, down, h, L.most_slices * a.row_tiles, st);
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
    a.row_tiles = (m.N + kNW - 1) / kNW;
    a.M = m.M;
    a.as = m.as;
    a.ldas = m.ldas;
    a.ws0 = m.bs;
    a.out = m.out;
    a.ldo = m.ldo;
    a.vec = (uintptr_t)m.out % 32 == 0 && m.ldo * dtype_bytes(m.dt) % 32 == 0 && m.N % 16 == 0;
    a.status = m.status;
    const int64_t tiles = (int64_t)((m.M + kMT - 1) / kMT) * a.row_tiles;
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
