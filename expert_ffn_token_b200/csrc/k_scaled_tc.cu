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
// and the 128 up rows of the same ffn values; 128 rows where a dense product has few tiles.
// Tokens sit on the M side so that a tensor-memory
// lane is a token: an epilogue thread's scale is then one number per block and operand.  With the
// weights on the M side the scale changes from column to column and has to be read from shared
// memory, two 16-byte loads per four elements; the loads, not the additions, then bound the
// kernel (1380 clocks per block of 128 k against 512 of MMA).  An expert with few tokens leaves
// rows of the MMA unused, which costs nothing that counts: it is bound by its weights' bytes.
//
// One persistent CTA per SM.  Pairs of CTAs (cta_group::2, 256 tokens a tile) load a third less per
// MMA, but the hand-overs between the two cost what the loads gain (side by side, before the
// epilogue's last steps: 8192^3 547 us against 560, 4096 x 1280 x 2560 37 against 35, 8192 routed
// tokens 1270 against 1006).  They are not used.
//
// Now, on the device: 8192^3 486 to 504 us back to back (2.2 PFLOP/s; 907 clocks a block of k, 512 of
// them its MMAs, with the issue slots 65 percent full, mostly of the sums' promotion), 4096 x 1280 x
// 2560 to fp32 30 us (160 tiles: two rounds).  The experts' layer of 10 of 512 experts and the shared
// one, hidden 2560, ffn 640: 64 tokens 303 us (5.9 TB/s of weights), 8192 tokens 910 to 940 us (to bf16).
//
// Roles (640 threads; registers move from the first four warps to the epilogue):
//   warp 0        TMA producer: weight boxes of 128 rows x 128 bytes, token rows as boxes of 16
//   warp 1        tensor-memory allocation and the MMA issuer
//   warp 2        the scales of every block, copied into a ring four blocks a hand-over
//   warps 4-19    epilogue: lane quarter (warp % 4), 32 columns of each 128-row operand.  Four warps
//                 a scheduler, because a block is a chain of hand-overs and tensor-memory loads
//                 that one warp cannot hide: with two, a block took 1250 clocks, 300 of them work
// Every hand-off is an mbarrier and every wait but the CTA's first and last __syncthreads, which
// all threads reach, is bounded (MOE_ERR_TIMEOUT in the status word; moe_scaled_set_wait_limit).
//
// The experts' layer quantises x straight into slot order, once per routed expert, so that every
// tile's token rows are neighbours.  Gathering them in this kernel cost more: a TMA gather of
// four rows takes about 70 clocks and a block needs 32, and one warp's 16-byte cp.async copies
// took 1.4 us a block where the loads of neighbouring rows take 0.5 us.
#include <algorithm>
#include <cstddef>

#include "route_dev.cuh"
#include "scaled.cuh"
#include "tc_pipe.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int kMT = kScaledRun;                // most tokens of a tile
constexpr int kNW = 256;                       // weight rows of a tile (gate/up: 128 + 128)
constexpr int kEpiWarp0 = 4, kEpiWarps = 16;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kOperand = 128 * kSBlk;     // bytes of 128 rows of one block
constexpr uint32_t kWeights = 2 * kOperand;    // a stage: the weights' two operands
constexpr uint32_t kStage = kWeights + kOperand;   // and the tokens
constexpr int kStages = 4;
constexpr int kAccs = 2;                       // accumulator buffers of 256 columns
constexpr int kBand = 8;                       // row tiles of a band (dense)
constexpr int kGroup = 4;                      // blocks whose scales are handed over together
constexpr int kScales = 4;                     // depth of the scale ring, in groups
constexpr int kPatch = 8;                      // columns per turn through shared memory (stores)
constexpr uint32_t kTmemCols = 512;
static_assert(kEpiWarps * 32 * 33 * 4 <= kStages * kStage, "the ring holds every warp's 32 columns");
constexpr uint64_t kDrainNs = 2000000000ull;   // limit of the waits for own copies and products
// Registers: 640 threads launch with 96 each (61440); the first warpgroup keeps 64 and the four
// epilogue warpgroups take 104: 128 * 64 + 512 * 104 = 61440.
constexpr int kLaunchRegs = 96, kRoleRegs = 64, kEpiRegs = 104;
static_assert(kAccs == 2, "the epilogue flips between two accumulators");
static_assert(sizeof(Job) == sizeof(int4), "a slice is loaded as one vector");
static_assert(128 * kRoleRegs + 512 * kEpiRegs <= kThreads * kLaunchRegs, "register split");

enum Mode { kGateUp, kDown, kDense, kNarrow };
constexpr bool dense(int mode) { return mode == kDense || mode == kNarrow; }
constexpr int operands(int mode) { return mode == kNarrow ? 1 : 2; }   // of 128 weight rows, a tile
constexpr int width(int mode) { return 128 * operands(mode); }

struct TcArgs {
    int nkb;                     // blocks of k
    int rows;                    // weight rows per expert (gate/up: of each of the two)
    int row_tiles;
    int M;                       // dense: rows of a
    const Job *slices;           // experts: runs of up to 128 slots (list_slices)
    const int32_t *nslices;
    const float *as;
    int64_t ldas;
    const float *ws0, *ws1;      // weight scales [expert][row blocks][nkb]; ws1: up
    int64_t ws_expert;
    uint8_t *hq;                 // gate/up: [slots][rows] and scales [row blocks][slots]
    float *hs;
    int64_t slots;
    uint8_t *ys;                 // down to fp16: powers of two [slots][32 columns], as fp32 exponents
    void *out;
    int64_t ldo;
    bool vec;                    // out rows are 32-byte aligned and rows a multiple of 16
    uint32_t *status;
    uint64_t wait_ns;            // limit of every hand-over's wait (moe_scaled_set_wait_limit)
    uint32_t look;               // the clock is looked at where a wait's tries have none of these bits
};

struct Tile {
    int e, rt, slot, n;
};

// Powers of two of y, one per 32 columns: a row tile's eight are neighbours, the two of a thread
// (columns c and c + 128) one 16-bit store.
__host__ __device__ inline int ypitch(int n) { return (n + kNW - 1) / kNW * 8; }
__device__ __forceinline__ int yindex(int c) { return c / kNW * 8 + c % 128 / 32 * 2 + c % kNW / 128; }

// Tile i.  Experts: row tiles are innermost, so that the CTAs that run at the same time share
// an expert's weights (its slices follow one another) and a slice's tokens.
template <int kMode>
__device__ __forceinline__ Tile tile_at(const TcArgs &a, int i) {
    Tile t;
    int s = i / a.row_tiles;
    t.rt = i - s * a.row_tiles;
    if (dense(kMode)) {
        // bands of kBand row tiles, so that the tiles in flight cover a compact part of both sides
        const int ns = (a.M + kMT - 1) / kMT;
        const int band = i / (kBand * ns), in = i - band * (kBand * ns);
        const int wide = min(kBand, a.row_tiles - band * kBand);
        s = in / wide;
        t.rt = band * kBand + in - s * wide;
        t.e = 0;
        t.slot = s * kMT;
        t.n = min(kMT, a.M - t.slot);
    } else {
        const int4 v = __ldg(reinterpret_cast<const int4 *>(a.slices) + s);
        t.e = v.x;
        t.slot = v.y;
        t.n = v.z;
    }
    return t;
}

struct Shared {
    uint64_t full[kStages], empty[kStages], acc_full[kAccs], acc_empty[kAccs], sc_full[kScales],
        sc_empty[kScales], quarter[4], done;
    uint32_t tmem;
    int abort;
    float as[kScales][kGroup][kMT];       // per block: the tokens' scales
    float2 ws[kScales][kGroup];           // and the two operands' weight scales
    uint32_t amax[2][4][kMT];             // gate/up: by tile parity and column quarter, per token
    float patch[kEpiWarps][32][kPatch + 1];
};

// Shared follows the ring, whose stages keep the 1024-byte alignment of its start; scales are copied
// 4 bytes at a time and the weights' read in pairs.
static_assert(kStage % 1024 == 0 && alignof(Shared) == 8 && offsetof(Shared, full) == 0 &&
                  offsetof(Shared, as) % 4 == 0 && offsetof(Shared, ws) % sizeof(float2) == 0 &&
                  sizeof(float2) == 8,
              "alignment of what the copies and vector loads touch");

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

// Bounded wait of a whole warp, with one answer: false once this CTA gives up.  The clock and the
// abort flag are looked at once in 64 tries: reading the global timer between tries would delay
// the wake-up.  A try suspends the warp for longer than a hand-over takes, so under a short limit
// the tries do not suspend and the clock is looked at after each.  The vote keeps the loop uniform.
__device__ __forceinline__ bool waitw(const TcArgs &a, Shared &S, uint64_t *bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_test_wait(bar, parity))) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(kFull, a.look ? mbar_try_wait(bar, parity)
                                                   : mbar_test_wait(bar, parity)); i++) {
        if (i & a.look) continue;
        const uint64_t t = globaltimer();
        if (t0 == 0) t0 = t;
        const bool late = t - t0 > a.wait_ns;
        if (late) {
            *(volatile int *)&S.abort = 1;
            set_status(a.status, MOE_ERR_TIMEOUT);
        }
        if (__any_sync(kFull, late || *(volatile int *)&S.abort)) return false;
    }
    return true;
}
// One arrival of the warp, without a branch.
__device__ __forceinline__ void arrive1(uint64_t *bar, bool mine) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"((uint32_t)mine)
        : "memory");
}

template <int kMode>
__device__ void produce(const TcArgs &a, Shared &S, uint8_t *ring, int tiles, const CUtensorMap *w0,
                        const CUtensorMap *w1, const CUtensorMap *x, const CUtensorMap *x16) {
    const int lane = threadIdx.x & 31;
    Pos p;
    int issued = 0;
    int i = blockIdx.x;
    if (i >= tiles) return;
    Tile next = tile_at<kMode>(a, i);
    bool ok = true;                   // until a wait runs out
    for (; ok && i < tiles; i += gridDim.x) {
        const Tile t = next;
        // more than half a tile of tokens comes as one box of 128 rows (those past the slice, if
        // they exist, are read and not used): every box costs the copy engine time of its own
        const bool whole = t.n > kMT / 2;
        const int npad = whole ? kMT : (t.n + 15) & ~15;
        // the next tile's place arrives while this one's blocks are issued
        if (i + (int)gridDim.x < tiles) next = tile_at<kMode>(a, i + gridDim.x);
        for (int b = 0; b < a.nkb; b++) {
            if (!waitw(a, S, &S.empty[p.s], p.ph ^ 1u)) {
                ok = false;
                break;
            }
            uint8_t *st = ring + (size_t)p.s * kStage;
            uint64_t *bar = &S.full[p.s];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, operands(kMode) * kOperand + (uint32_t)npad * kSBlk);
                const int r0 = kMode == kGateUp ? t.rt * 128 : t.rt * width(kMode);
                const int r1 = kMode == kGateUp ? r0 : r0 + 128;
                tma_load_3d(st, w0, b * kSBlk, r0, t.e, bar);
                if (operands(kMode) == 2) tma_load_3d(st + kOperand, w1, b * kSBlk, r1, t.e, bar);
                if (whole) tma_load_2d(st + kWeights, x, b * kSBlk, t.slot, bar);
            }
            __syncwarp();
            if (!whole && 16 * lane < npad)
                tma_load_2d(st + kWeights + lane * 16 * kSBlk, x16, b * kSBlk, t.slot + 16 * lane,
                            bar);
            issued++;
            p.next(kStages);
        }
    }
    // whoever gives up: the copies in flight land before the CTA goes
    for (int j = max(0, issued - kStages); j < issued; j++)
        mbar_wait_bounded(&S.full[j % kStages], (uint32_t)(j / kStages) & 1u, kDrainNs);
}

// Blocks of the tiles that this CTA takes.
__device__ __forceinline__ int64_t blocks_of_cta(const TcArgs &a, int tiles) {
    const int step = gridDim.x;
    return (int64_t)(max(0, tiles - (int)blockIdx.x + step - 1) / step) * a.nkb;
}

// The MMA issuer.  The whole warp walks the loop and one elected lane issues, so that the
// descriptors stay in uniform registers.
template <int kMode>
__device__ void multiply(const TcArgs &a, Shared &S, uint8_t *ring, int tiles, uint32_t tmem) {
    constexpr uint32_t idesc = instr_desc(0, kMT, width(kMode));
    const int64_t total = blocks_of_cta(a, tiles);
    Pos p, q;
    for (int64_t i = 0; i < total; i++) {
        if (!waitw(a, S, &S.full[p.s], p.ph) ||
            !waitw(a, S, &S.acc_empty[q.s], q.ph ^ 1u))
            break;
        tc_fence_after();
        const uint32_t st = smem_u32(ring) + (uint32_t)p.s * kStage;
        const uint64_t x = smem_desc(st + kWeights, 1024, 2), w = smem_desc(st, 1024, 2);
        const uint32_t d = tmem + (uint32_t)(q.s * kNW);
        if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; j++)          // 32 bytes of k a step: 2 units of 16 bytes
                umma_f8(d, x + 2 * j, w + 2 * j, idesc, j > 0);
            umma_commit(&S.acc_full[q.s]);
            umma_commit(&S.empty[p.s]);
        }
        __syncwarp();
        p.next(kStages);
        q.next(kAccs);
    }
    // whoever gives up: no MMA is in flight when the tensor memory goes
    if (elect_one()) {
        umma_commit(&S.done);
        mbar_wait_bounded(&S.done, 0, kDrainNs);
    }
    __syncwarp();
}

// Warp 2: the scales of every block, in the order the epilogue takes them, copied into the ring.
template <int kMode>
__device__ void scales(const TcArgs &a, Shared &S, int tiles) {
    const int lane = threadIdx.x & 31;
    Pos p;
    int u = 0;                              // block within the group
    int i = blockIdx.x;
    if (i >= tiles) return;
    Tile next = tile_at<kMode>(a, i);
    for (; i < tiles; i += gridDim.x) {
        const Tile t = next;
        const float *as = a.as + t.slot + lane;
        const float *s0 = a.ws0 + t.e * a.ws_expert, *s1;
        if (kMode == kGateUp) {
            s0 += (int64_t)t.rt * a.nkb;
            s1 = a.ws1 + t.e * a.ws_expert + (int64_t)t.rt * a.nkb;
        } else {
            s0 += (int64_t)(operands(kMode) * t.rt) * a.nkb;
            // past the last rows: not stored
            s1 = operands(kMode) == 2 && t.rt * kNW + kSBlk < a.rows ? s0 + a.nkb : s0;
        }
        const float *mine_ws = lane == 0 ? s0 : s1;
        if (i + (int)gridDim.x < tiles) next = tile_at<kMode>(a, i + gridDim.x);
#pragma unroll 1
        for (int b = 0; b < a.nkb; b++) {
            if (u == 0 && !waitw(a, S, &S.sc_empty[p.s], p.ph ^ 1u)) {
                cp_async_wait_all();
                return;
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (lane + 32 * j < t.n) cp_async4(&S.as[p.s][u][lane + 32 * j], as + 32 * j);
            if (lane < 2)
                cp_async4(reinterpret_cast<float *>(&S.ws[p.s][u]) + lane, mine_ws + b);
            as += a.ldas;
            if (++u == kGroup) {
                u = 0;
                cp_async_arrive(&S.sc_full[p.s]);
                p.next(kScales);
            }
        }
    }
    if (u) cp_async_arrive(&S.sc_full[p.s]);
    cp_async_wait_all();                    // the epilogue may have given up on them
}

// acc += r * s for 16 columns.  (Packed two-element multiply-adds need the loaded registers in
// pairs; the moves that pairs them cost more than the halved instruction count gains.)
__device__ __forceinline__ void promote16(float *acc, const uint32_t (&r)[16], float s) {
#pragma unroll
    for (int i = 0; i < 16; i++) acc[i] = fmaf(__uint_as_float(r[i]), s, acc[i]);
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

// 16 columns of this lane's row at p, 32-byte aligned.
template <typename T>
__device__ __forceinline__ void store16(T *p, const float *acc) {
    uint32_t v[8];
    if (sizeof(T) == 4) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = __float_as_uint(acc[8 * h + i]);
            store32B(p + 8 * h, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = pack2(acc[2 * i], acc[2 * i + 1], (T *)nullptr);
        store32B(p, v);
    }
}

template <int kMode, typename T>
__device__ void finish(const TcArgs &a, Shared &S, uint8_t *ring, int tiles, uint32_t tmem) {
    const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int quad = warp & 3, part = (warp - kEpiWarp0) >> 2;
    const int row = quad * 32 + lane;
    constexpr bool kHalfY = kMode == kDown && sizeof(T) == 2;   // y in fp16
    const uint32_t base = tmem + ((uint32_t)quad << 21) + (uint32_t)(part * 32);  // lane quad * 32
    uint32_t q = 0, qph = 0;            // accumulator and its phase
    Pos p;
    int u = 0;                          // block within the scale ring's group
    uint32_t par = 0;
    int i = blockIdx.x;
    if (i >= tiles) return;
    Tile next = tile_at<kMode>(a, i);
    for (; i < tiles; i += gridDim.x) {
        const Tile t = next;
        if (i + (int)gridDim.x < tiles) next = tile_at<kMode>(a, i + gridDim.x);
        float acc[2][32];
#pragma unroll
        for (int j = 0; j < 32; j++) acc[0][j] = acc[1][j] = 0.f;
        const bool busy = quad * 32 < t.n;
#pragma unroll 1
        for (int b = 0; b < a.nkb; b++) {
            if (u == 0 && !waitw(a, S, &S.sc_full[p.s], p.ph)) return;
            const float v = S.as[p.s][u][row];
            const float2 w = S.ws[p.s][u];
            if (!waitw(a, S, &S.acc_full[q], qph)) return;
            if (busy) {
                const float f[2] = {v * w.x, v * w.y};
                tc_fence_after();
                const uint32_t d = base + q * kNW;
#pragma unroll
                for (int o = 0; o < operands(kMode); o++) {
#pragma unroll
                    for (int j = 0; j < 32; j += 16) {
                        uint32_t r[16];
                        tmem_ld16(d + o * 128 + j, r);
                        tmem_ld_wait(r);
                        promote16(acc[o] + j, r, f[o]);
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            arrive1(&S.acc_empty[q], lane == 0);
            qph ^= q;                            // after the second accumulator
            q ^= 1u;
            if (++u == kGroup) {
                u = 0;
                arrive1(&S.sc_empty[p.s], lane == 0);
                p.next(kScales);
            }
        }
        if (!busy) continue;
        if (kMode == kGateUp) {
            // h, and its e4m3 form per token and 128 ffn values: this thread's 32 and those of the
            // other three column quarters
            bool far = false;
#pragma unroll
            for (int j = 0; j < 32; j++) far |= acc[0][j] < kSiluFar;
            if (far && row < t.n) {
#pragma unroll
                for (int j = 0; j < 32; j++) acc[0][j] = swiglu(acc[0][j], acc[1][j]);
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++) acc[0][j] = swiglu_near(acc[0][j], acc[1][j]);
            }
            uint32_t mx = 0u;
#pragma unroll
            for (int j = 0; j < 32; j++) mx = max(mx, __float_as_uint(acc[0][j]) & 0x7fffffffu);
            S.amax[par][part][row] = mx;
            // the quarter's four warps meet at an mbarrier: a warp that gave up must not hold the others
            __syncwarp();
            arrive1(&S.quarter[quad], lane == 0);
            if (!waitw(a, S, &S.quarter[quad], par)) return;
            mx = max(max(S.amax[par][0][row], S.amax[par][1][row]),
                     max(S.amax[par][2][row], S.amax[par][3][row]));
            par ^= 1u;
            if (row < t.n) {
                const bool fin = mx < 0x7f800000u;
                const float sc = fin ? __fdiv_rn(__uint_as_float(mx), kE4M3Max) : 0.f;
                // both sides of h / sc times 2^100, exactly, where a tiny scale has no reciprocal
                float s = sc;
                if (sc < 0x1p-100f) {
                    s *= 0x1p100f;
#pragma unroll
                    for (int j = 0; j < 32; j++) acc[0][j] *= 0x1p100f;
                }
                const float inv = __frcp_rn(s);
                const int64_t slot = (int64_t)t.slot + row;
                if (part == 0) {
                    a.hs[t.rt * a.slots + slot] = sc;
                    if (!fin) set_status(a.status, MOE_ERR_NONFINITE);
                }
                const int f = t.rt * 128 + part * 32;
                uint8_t *hq = a.hq + slot * a.rows + f;
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    uint32_t v[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const float *x = acc[0] + 16 * j + 4 * u;
                        v[u] = quant4_normal(make_float4(x[0], x[1], x[2], x[3]), s, inv);
                        if (!(sc > 0.f)) v[u] = 0u;
                    }
                    if (f + 16 * j < a.rows)
                        *reinterpret_cast<uint4 *>(hq + 16 * j) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        } else {
            T *out = static_cast<T *>(a.out) + ((int64_t)t.slot + row) * a.ldo;
            uint32_t ex = 0u;
#pragma unroll
            for (int u = 0; u < operands(kMode); u++) {
                const int r0 = t.rt * width(kMode) + u * 128 + part * 32;
                if (kHalfY) {
                    // y as fp16 times a power of two per token and 32 columns, which are this thread's:
                    // the largest magnitude goes to [2^14, 2^15), so that what rounds as a
                    // subnormal is 2^28 times smaller
                    float mx = 0.f;                    // (passes over NaN, which stays NaN)
#pragma unroll
                    for (int j = 0; j < 32; j++) mx = fmaxf(mx, fabsf(acc[u][j]));
                    if (mx == INFINITY && row < t.n) {     // which stays too: the others count
                        mx = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            if (fabsf(acc[u][j]) < INFINITY) mx = fmaxf(mx, fabsf(acc[u][j]));
                    }
                    // at most 113
                    const int x = max((int)(__float_as_uint(mx) >> 23) - 127 - 14, -126);
                    const float inv = __uint_as_float((uint32_t)(127 - x) << 23);
                    ex |= (uint32_t)(127 + x) << (8 * u);
                    if (u == 1 && row < t.n)
                        *reinterpret_cast<uint16_t *>(a.ys + ((int64_t)t.slot + row) * ypitch(a.rows) +
                                                      8 * t.rt + 2 * part) = (uint16_t)ex;
#pragma unroll
                    for (int j = 0; j < 32; j++) acc[u][j] *= inv;
                }
                if (a.vec) {
                    // 32 bytes of a row per lane and store
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        if (row < t.n && r0 + 16 * j < a.rows)
                            store16(out + r0 + 16 * j, acc[u] + 16 * j);
                } else {
                    // rows of any alignment, through shared memory, so that a warp writes runs of a
                    // row: after this CTA's last tile 32 columns at a time in the operand ring,
                    // which no copy or MMA uses any more, before that 8 in a patch of its own
                    // (777 x 1001 x 1296, one wide tile per CTA, on the device: 12.9 us, with the patch 14.8).
                    // Every MMA is over by then: the wait for the last block's sums was for all of them
                    const bool last = i + (int)gridDim.x >= tiles;
                    const int run = last ? 32 : kPatch, pitch = run + 1;
                    float *P = last ? reinterpret_cast<float *>(ring) + (warp - kEpiWarp0) * 32 * 33
                                    : &S.patch[warp - kEpiWarp0][0][0];
                    const int first = lane / run, step = 32 / run, col = lane % run;
#pragma unroll
                    for (int j = 0; j < 32 / kPatch; j++) {
#pragma unroll
                        for (int x = 0; x < kPatch; x++)
                            P[lane * pitch + x + (last ? kPatch * j : 0)] = acc[u][kPatch * j + x];
                        if (last && j + 1 < 32 / kPatch) continue;
                        __syncwarp();
                        const int c = r0 + (last ? 0 : kPatch * j) + col;
                        T *o = static_cast<T *>(a.out) +
                               ((int64_t)t.slot + quad * 32 + first) * a.ldo + c;
                        if (c < a.rows) {
                            const int most = min(32, t.n - quad * 32);
#pragma unroll 4
                            for (int y = first; y < most; y += step, o += step * a.ldo)
                                *o = from_f32<T>(P[y * pitch + col]);
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
                const __grid_constant__ CUtensorMap w1, const __grid_constant__ CUtensorMap x,
                const __grid_constant__ CUtensorMap x16) {
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Shared &S = *reinterpret_cast<Shared *>(ring + (size_t)kStages * kStage);
    const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0);
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
            mbar_init(&S.sc_full[i], 32);
            mbar_init(&S.sc_empty[i], kEpiWarps);
        }
        for (int i = 0; i < 4; i++) mbar_init(&S.quarter[i], 4);
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
    const int tiles = (dense(kMode) ? (a.M + kMT - 1) / kMT : *a.nslices) * a.row_tiles;
    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
        if (warp == 0)
            produce<kMode>(a, S, ring, tiles, &w0, &w1, &x, &x16);
        else if (warp == 1)
            multiply<kMode>(a, S, ring, tiles, tmem);
        else if (warp == 2)
            scales<kMode>(a, S, tiles);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        finish<kMode, T>(a, S, ring, tiles, tmem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Eight values of y at column 8 c of a slot's row, with their power of two when y is fp16.
__device__ __forceinline__ void load_y(const float *y, const uint8_t *, int64_t slot, int H, int c,
                                       float (&v)[8]) {
    const float4 *p = reinterpret_cast<const float4 *>(y + slot * H) + 2 * c;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load_y(const __half *y, const uint8_t *ys, int64_t slot, int H, int c,
                                       float (&v)[8]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(y + slot * H) + c);
    const float s = __uint_as_float((uint32_t)__ldg(ys + slot * ypitch(H) + yindex(8 * c)) << 23);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

// out[t] = sum_j w[t][j] y[slot of (t, j)] (+ gate[t] y[routed + t]), in the order of j.  A warp
// takes 256 columns of a token, eight per lane; reads y once: bound by memory.
template <typename Y, typename T>
__global__ void __launch_bounds__(256)
    k_scaled_combine(const Y *__restrict__ y, const uint8_t *__restrict__ ys,
                     const int32_t *__restrict__ inv_perm, const int32_t *__restrict__ ids,
                     const float *__restrict__ w, const float *__restrict__ gate, int tokens,
                     int k, int E, int shared, int H, T *__restrict__ out, uint32_t *status) {
    const int lane = threadIdx.x & 31;
    const int per = (H / 8 + 31) / 32;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t t = unit / per;
    if (t >= tokens) return;
    const int c = (int)(unit - t * per) * 32 + lane;
    const int A = tokens * k;
    // lane j holds pair j's slot and weight
    int slot = -1;
    float wt = 0.f;
    if (lane < k) {
        const int s = __ldg(inv_perm + t * k + lane), e = __ldg(ids + t * k + lane);
        const bool in = s >= 0 && s < A && e >= 0 && e < E;
        if (!in) set_status(status, MOE_ERR_BOUNDS);
        slot = in ? s : -1;
        wt = __ldg(w + t * k + lane);
    }
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] = 0.f;
    const bool in = 8 * c < H;
#pragma unroll 4
    for (int j = 0; j < k; j++) {
        const int s = __shfl_sync(kFull, slot, j);
        const float f = __shfl_sync(kFull, wt, j);
        if (s < 0 || !in) continue;
        float v[8];
        load_y(y, ys, s, H, c, v);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = fmaf(f, v[i], acc[i]);
    }
    if (!in) return;
    if (shared) {
        const float f = gate ? __ldg(gate + t) : 1.0f;
        float v[8];
        load_y(y, ys, (int64_t)A + t, H, c, v);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = fmaf(f, v[i], acc[i]);
    }
    T *o = out + t * H + 8 * c;
    if (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(o)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        reinterpret_cast<float4 *>(o)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
        *reinterpret_cast<uint4 *>(o) =
            make_uint4(pack2(acc[0], acc[1], (T *)nullptr), pack2(acc[2], acc[3], (T *)nullptr),
                       pack2(acc[4], acc[5], (T *)nullptr), pack2(acc[6], acc[7], (T *)nullptr));
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

void set_limit(TcArgs &a, uint64_t ns) {
    a.wait_ns = ns;
    a.look = ns < 1000000 ? 0 : 63;
}

template <int kMode, typename T>
cudaError_t run_tc(const TcArgs &a, const CUtensorMap &w0, const CUtensorMap &w1,
                   const CUtensorMap &x, const CUtensorMap &x16, int64_t most_tiles,
                   cudaStream_t st) {
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
    kernel<<<(unsigned)std::min<int64_t>(sms, most_tiles), kThreads, kSmem, st>>>(a, w0, w1, x, x16);
    note_launches(1);
    return cudaGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct ExpertsWs {
    size_t xq, xs, hq, hs, y, ys, slices, nslices, total;
    int64_t slots, most_slices;
};

// y is sized for fp32; with a bf16 output it is fp16.
ExpertsWs experts_ws(const moe_scaled_weights &w, int T, int k) {
    ExpertsWs L{};
    size_t p = 0;
    auto take = [&](size_t bytes) {
        const size_t o = p;
        p = align256(p + bytes);
        return o;
    };
    L.slots = (int64_t)T * k + (w.shared ? T : 0);
    L.xq = take((size_t)L.slots * w.hidden);
    L.xs = take((size_t)sblocks(w.hidden) * L.slots * 4);
    L.hq = take((size_t)L.slots * w.ffn);
    L.hs = take((size_t)sblocks(w.ffn) * L.slots * 4);
    L.y = take((size_t)L.slots * w.hidden * 4);
    L.ys = take((size_t)L.slots * ypitch(w.hidden));
    L.most_slices = (int64_t)T * k / kMT + std::min<int64_t>(w.n_experts, (int64_t)T * k) +
                    (w.shared ? (T + kMT - 1) / kMT : 0);
    L.slices = take(sizeof(Job) * (size_t)L.most_slices);
    L.nslices = take(4);
    L.total = p;
    return L;
}

template <typename Y, typename E>
cudaError_t run_combine(const ScaledExpertsArgs &e, const void *y, const uint8_t *ys, cudaStream_t st) {
    const moe_scaled_weights &w = e.w;
    const int64_t units = (int64_t)e.T * ((w.hidden / 8 + 31) / 32);
    k_scaled_combine<Y, E><<<(unsigned)((units + 7) / 8), 256, 0, st>>>(
        static_cast<const Y *>(y), ys, e.inv_perm, e.ids, e.rw, e.gate, e.T, e.k, w.n_experts,
        w.shared, w.hidden, static_cast<E *>(e.out), e.status);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t experts_tc(const ScaledExpertsArgs &e, uint8_t *ws, cudaStream_t st) {
    const moe_scaled_weights &w = e.w;
    const ExpertsWs L = experts_ws(w, e.T, e.k);
    const int n = w.n_experts + w.shared, H = w.hidden, F = w.ffn;
    Job *slices = reinterpret_cast<Job *>(ws + L.slices);
    int32_t *nslices = reinterpret_cast<int32_t *>(ws + L.nslices);
    float *xs = reinterpret_cast<float *>(ws + L.xs);
    uint8_t *ys = ws + L.ys;
    CUtensorMap gate, up, down, x, x16, h, h16;
    if (!encode(&gate, w.d_gate, H, F, H, n, 128) || !encode(&up, w.d_up, H, F, H, n, 128) ||
        !encode(&down, w.d_down, F, H, F, n, 128) ||
        !encode(&x, ws + L.xq, H, L.slots, H, 0, 128) ||
        !encode(&x16, ws + L.xq, H, L.slots, H, 0, 16) ||
        !encode(&h, ws + L.hq, F, L.slots, F, 0, 128) ||
        !encode(&h16, ws + L.hq, F, L.slots, F, 0, 16))
        return cudaErrorInvalidValue;
    cudaError_t err = launch_scaled_spread(e, ws + L.xq, xs, slices, nslices, st);
    if (err != cudaSuccess) return err;
    TcArgs a{};
    a.slices = slices;
    a.nslices = nslices;
    a.status = e.status;
    set_limit(a, e.wait_ns);
    a.slots = L.slots;
    a.hq = ws + L.hq;
    a.hs = reinterpret_cast<float *>(ws + L.hs);
    a.nkb = sblocks(H);
    a.rows = F;
    a.row_tiles = sblocks(F);
    a.as = xs;
    a.ldas = L.slots;
    a.ws0 = w.d_gate_s;
    a.ws1 = w.d_up_s;
    a.ws_expert = (int64_t)sblocks(F) * sblocks(H);
    err = run_tc<kGateUp, float>(a, gate, up, x, x16, L.most_slices * a.row_tiles, st);
    if (err != cudaSuccess) return err;
    a.nkb = sblocks(F);
    a.rows = H;
    a.row_tiles = (H + kNW - 1) / kNW;
    a.as = a.hs;
    a.ws0 = w.d_down_s;
    a.out = ws + L.y;
    a.ldo = H;
    a.vec = true;
    const int64_t tiles = L.most_slices * a.row_tiles;
    // y is fp32, but for a bf16 output: there fp16's rounding is an eighth of the output's own, and
    // half the bytes are written and read.  For an fp16 output the two would be equal.
    if (e.out_dt != MOE_DT_BF16) {
        err = run_tc<kDown, float>(a, down, down, h, h16, tiles, st);
        if (err != cudaSuccess) return err;
        return e.out_dt == MOE_DT_F32 ? run_combine<float, float>(e, ws + L.y, nullptr, st)
                                      : run_combine<float, __half>(e, ws + L.y, nullptr, st);
    }
    a.ys = ys;
    err = run_tc<kDown, __half>(a, down, down, h, h16, tiles, st);
    return err != cudaSuccess ? err : run_combine<__half, __nv_bfloat16>(e, ws + L.y, ys, st);
}

cudaError_t matmul_tc(const ScaledMatmulArgs &m, cudaStream_t st) {
    CUtensorMap b, x, x16;
    if (!encode(&b, m.b, m.K, m.N, m.ldb, 1, 128) || !encode(&x, m.a, m.K, m.M, m.lda, 0, 128) ||
        !encode(&x16, m.a, m.K, m.M, m.lda, 0, 16))
        return cudaErrorInvalidValue;
    TcArgs a{};
    a.nkb = sblocks(m.K);
    a.rows = m.N;
    a.M = m.M;
    a.as = m.as;
    a.ldas = m.ldas;
    a.ws0 = m.bs;
    a.out = m.out;
    a.ldo = m.ldo;
    a.vec = (uintptr_t)m.out % 32 == 0 && m.ldo * dtype_bytes(m.dt) % 32 == 0 && m.N % 16 == 0;
    a.status = m.status;
    set_limit(a, m.wait_ns);
    const int64_t ms = (m.M + kMT - 1) / kMT;
    const int64_t sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Tiles of 128 weight rows where all of them run at once: 777 x 1001 x 1296 9.5 us (wide 13.6),
    // 1024 x 1280 x 2560 11.6 (13.8).  Past that wide ones: a narrow tile takes 70 percent of a
    // wide one's time, so 2048 x 1280 x 2560 19.6 us (wide 14.3), 8192 x 4096 x 4096 180 (133).
    const bool narrow = ms * ((m.N + 127) / 128) <= sms;
    const int w = narrow ? width(kNarrow) : width(kDense);
    a.row_tiles = (m.N + w - 1) / w;
    const int64_t tiles = ms * a.row_tiles;
    if (tiles > (1 << 30)) return cudaErrorInvalidValue;      // a tile index plus the grid fits
    return with_dtype(m.dt, [&](auto *tag) {
        using E = std::remove_pointer_t<decltype(tag)>;
        return narrow ? run_tc<kNarrow, E>(a, b, b, x, x16, tiles, st)
                      : run_tc<kDense, E>(a, b, b, x, x16, tiles, st);
    });
}

}  // namespace

size_t scaled_matmul_ws_bytes(int, int, int) { return 0; }

cudaError_t launch_scaled_matmul(const ScaledMatmulArgs &a, void *, cudaStream_t st) {
    return a.M <= kSmallT ? launch_scaled_small(a, st) : matmul_tc(a, st);
}

size_t scaled_experts_ws_bytes(const moe_scaled_weights &w, int T, int k) {
    return T <= kSmallExpertsT ? align256(scaled_small_ws_bytes(T, k, w.shared, w.hidden, w.ffn))
                        : experts_ws(w, T, k).total;
}

cudaError_t launch_scaled_experts(const ScaledExpertsArgs &a, void *ws, cudaStream_t st) {
    return a.T > kSmallExpertsT ? experts_tc(a, static_cast<uint8_t *>(ws), st)
                         : launch_scaled_experts_small(a, ws, st);
}

}  // namespace moe
