// bwd_bf16_sm103.cu -- ring-attention backward for sm_103a tensor cores.
//
// The pages state only that context parallelism leaves the gradients equal to
// single-device training ("Sequence and Context Parallelism", "What it does
// not change") and that activations are kept for the backward pass ("Sequence
// Parallelism in LLMs", "The Activation Memory Wall"); they give no backward
// algorithm.  This file computes the textbook gradient of attention with the
// saved lse, over the same (rank, ring step, tile) schedule as the forward:
//   P = exp(scale * q k^T - lse)   (masked by global positions)
//   Delta_i = rowsum(dO_i * out_i)
//   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - Delta)
//   dQ = scale * dS K,  dK = scale * dS^T Q
//
// Three launches:
//   bwd_delta  -- Delta (fp32) into the caller's workspace (HBM-bound).
//   bwd_dq     -- query-stationary: per 128-row query tile, walk the KV tiles
//                 of every ring step (as the forward does), S = Q K^T and
//                 dP = dO V^T into tensor memory, dS in bf16 back into tensor
//                 memory, dQ += dS K accumulated in tensor memory.
//   bwd_dkdv   -- key-stationary: per 128-key tile, walk the query tiles of
//                 every rank that holds it at some ring step, S^T = K Q^T and
//                 dP^T = V dO^T into tensor memory, P^T and dS^T in bf16 back
//                 into tensor memory, dV += P^T dO and dK += dS^T Q.
// Splitting dQ from dK/dV recomputes S and dP once more (7 tile MMAs per
// visible tile pair instead of 5) but needs no atomics: every output element
// is written once, and the result is deterministic.
//
// Roles of both tensor-core kernels (384 threads, three warpgroups): warp 0
// TMA producer (dQ: K tiles; warp 3 loads Q, dO and V), MMA issuers that run
// converged with one elected lane issuing (dQ: warps 1 and 2; dK/dV: warps 1,
// 2 and 3), warps 4-7 and 8-11 the elementwise gradient (dQ: the two
// 64-column halves of one 128x128 tile; dK/dV: one warpgroup per half-step
// buffer), one thread per tensor-memory lane.  Every wait is bounded.
//
// WIN: the gradients of windowed attention with sinks (window_attn_bwd), by the same
// formulas over its visible pairs: WinIter's walk for dQ, WinQIter's for dK/dV, where the
// rows behind the window of a tile of sinks come in pieces (SinkPlan) whose partial sums
// window_sinks.cuh adds up.  Units are short (a window of 1024 is 9 or 10 tiles), so one
// block an SM takes them in turn, its barriers' phases running on, and a unit's loads and
// first products go beside the end of the one before.  Delta is made by the dQ kernel.
// Bounded by the tensor cores and, in half of the time, by the chains at the ends of units
// and the latency of the elementwise part: 16384 rows, 16 heads, D = 128, window 1024 and 4
// sinks 202 us for dQ with Delta and 270 for dK/dV (187 and 247 without sinks); whole causal
// attention of that size at 1.38 and 1.32 PFLOP/s of the products made.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "cp_common.cuh"
#include "kernels.h"
#include "tc_helpers.cuh"
#include "tmem_io.cuh"
#include "window_fix.cuh"
#include "window_sinks.cuh"

namespace cp {

namespace {

using namespace tc;

constexpr int T = 128;             // tile rows (queries or keys)
constexpr int NTHREADS = 384;
constexpr int REGS_CTRL = 88;
constexpr int REGS_GRAD = 208;
static_assert(128 * REGS_CTRL + 256 * REGS_GRAD <= NTHREADS * 168, "register split exceeds the launch budget");
constexpr float LOG2E = 1.4426950408889634f;

template <int D>
struct Tile {
    static constexpr int BOXES = D / 64;
    static constexpr int BOX = 128 * 128;
    static constexpr int BYTES = BOXES * BOX;
};

// Unrolled issue sequences (compile-time offsets added to base descriptors
// inside the MMA asm): the MMA threads share their SM sub-partitions with busy
// gradient warps, so they spend as few instructions per MMA as possible.

// D/16 MMAs M=128, K=16, A and B K-major; A in 128-row boxes (16 KB), B in
// boxes of BOXB bytes (16 KB for 128 rows, 8 KB for 64)
template <int KK, int D, int BOXB>
__device__ __forceinline__ void ss_seq(uint32_t tD, uint64_t dA, uint64_t dB, uint32_t id)
{
    if constexpr (KK < D / 16) {
        constexpr uint32_t oa = (uint32_t)(((KK >> 2) * 16384 + (KK & 3) * 32) >> 4);
        constexpr uint32_t ob = (uint32_t)(((KK >> 2) * BOXB + (KK & 3) * 32) >> 4);
        mma_ss_off<oa, ob>(tD, dA, dB, id, KK > 0 ? 1u : 0u);
        ss_seq<KK + 1, D, BOXB>(tD, dA, dB, id);
    }
}

// D/16 MMAs M=128, K=16: A (bf16 pairs, 8 columns per 16 elements) from tensor
// memory, B K-major in 128-row boxes (16 KB)
template <int KK, int D>
__device__ __forceinline__ void ts_k_seq(uint32_t tD, uint32_t tA, uint64_t dB, uint32_t id)
{
    if constexpr (KK < D / 16) {
        constexpr uint32_t ob = (uint32_t)(((KK >> 2) * 16384 + (KK & 3) * 32) >> 4);
        mma_ts_off<ob>(tD, tA + (uint32_t)(KK * 8), dB, id, KK > 0 ? 1u : 0u);
        ts_k_seq<KK + 1, D>(tD, tA, dB, id);
    }
}

// NK MMAs M=128, N=D, K=16: A (bf16 pairs) from tensor memory, B MN-major
// (k-steps of 16 rows, 2048 B); A columns relative to tA: 8 KK (MAP 0), or
// 32 (KK/2) + 8 (KK%2) (MAP 1: two runs of 16 columns, 32 apart).
// acc0 = accumulate flag of the first MMA.
template <int KK, int NK, int MAP>
__device__ __forceinline__ void ts_mn_seq(uint32_t tD, uint32_t tA, uint64_t dB, uint32_t id,
                                          uint32_t acc0)
{
    if constexpr (KK < NK) {
        constexpr uint32_t acol = MAP == 0 ? (uint32_t)(KK * 8) : (uint32_t)(32 * (KK >> 1) + 8 * (KK & 1));
        constexpr uint32_t ob = (uint32_t)((KK * 2048) >> 4);
        mma_ts_off<ob>(tD, tA + acol, dB, id, KK == 0 ? acc0 : 1u);
        ts_mn_seq<KK + 1, NK, MAP>(tD, tA, dB, id, acc0);
    }
}

// NaN where one of 32 columns is not finite, else 0.
__device__ __forceinline__ float odd_columns(const uint32_t (&o)[32])
{
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) ffma2v(a, b, __uint_as_float(o[e]), __uint_as_float(o[e + 1]), 0.f, 0.f, a, b);
    return a + b;
}

// 32 columns of the lane's row times f, as bf16, to 32-byte aligned memory: regrouped, so
// that a store covers whole pieces of 64 bytes.  (Every lane its own row in 16 bytes took
// the dK / dV epilogue of a unit 5500 cycles, as long as three of its half steps.)
__device__ __forceinline__ void put_row_piece(__nv_bfloat16 *piece, bool ok, const uint32_t (&o)[32], float f, int lane)
{
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) pk[e] = pack_bf16(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
    store_warp_rows<16>(piece, ok, pk, lane);
}

// 32 bytes of a row, zeros where it is not there; rows32: 32-byte aligned.
__device__ __forceinline__ void load_chunk(const __nv_bfloat16 *p, bool there, bool rows32, uint32_t (&w)[8])
{
    if (there && rows32) {
        ld_global_v8u(p, w);
        return;
    }
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (there) x = reinterpret_cast<const uint4 *>(p)[0], y = reinterpret_cast<const uint4 *>(p)[1];
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
}

// ----------------------------------------------------------------------------- Delta

__global__ void __launch_bounds__(256) bwd_delta_kernel(const __nv_bfloat16 *__restrict__ out,
                                                        const __nv_bfloat16 *__restrict__ dout,
                                                        float *__restrict__ delta, int S, int Hq,
                                                        int D, int64_t rows)
{
    // one warp per (b, s, h) row, rows in BSHD order, ROWS of them at a time (one at a
    // time left the loads' latency exposed: 268 MB in 58 us)
    constexpr int ROWS = 4;
    const int lane = threadIdx.x & 31;
    const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t nw = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t r0 = wid * ROWS; r0 < rows; r0 += nw * ROWS) {
        float acc[ROWS];
        uint2 ov[ROWS], gv[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            ov[i] = gv[i] = make_uint2(0, 0);
            acc[i] = 0.f;
            if (r0 + i < rows && lane * 4 < D) {
                ov[i] = *reinterpret_cast<const uint2 *>(out + (r0 + i) * D + lane * 4);
                gv[i] = *reinterpret_cast<const uint2 *>(dout + (r0 + i) * D + lane * 4);
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const __nv_bfloat162 *o2 = reinterpret_cast<const __nv_bfloat162 *>(&ov[i]);
            const __nv_bfloat162 *g2 = reinterpret_cast<const __nv_bfloat162 *>(&gv[i]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 a = __bfloat1622float2(o2[e]);
                const float2 b = __bfloat1622float2(g2[e]);
                acc[i] = fmaf(a.x, b.x, acc[i]);
                acc[i] = fmaf(a.y, b.y, acc[i]);
            }
        }
#pragma unroll
        for (int off = 16; off; off >>= 1)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
        // lane i writes row i's
        float mine = acc[0];
#pragma unroll
        for (int i = 1; i < ROWS; ++i) mine = lane == i ? acc[i] : mine;
        const int64_t r = r0 + lane;
        if (lane < ROWS && r < rows) {
            int64_t h, b, s;
            if (rows >> 31 == 0) {   // 64-bit divisions took 1.3 of 29.6 us
                const unsigned bs = (unsigned)r / (unsigned)Hq, bb = bs / (unsigned)S;   // b * S + s
                h = (unsigned)r - bs * (unsigned)Hq;
                b = bb;
                s = bs - bb * (unsigned)S;
            } else {
                const int64_t bs = r / Hq;
                h = r % Hq;
                b = bs / S;
                s = bs % S;
            }
            delta[(b * Hq + h) * S + s] = mine;
        }
    }
}

// ----------------------------------------------------------------------------- dQ
//
// Query-stationary.  Tensor memory (columns): S [0,128), dP [128,256), the dQ
// accumulator [256, 256+D), dS in bf16 pairs [256+D, 320+D), the block's dO
// rows in bf16 pairs [320+D, 320+3D/2).  Shared memory holds the Q tile, four
// K stages and two V stages.  S = Q K^T reads both operands from shared
// memory; dP = dO V^T and dQ += dS K read their A operands from tensor memory
// (dO written there once by the gradient warps, dS on every tile), which
// halves the shared-memory reads of the dP MMAs.
//
// S(j) and dP(j) have their own barriers both ways, so S(j+1) is issued as
// soon as the gradient warps have read S(j) and runs while they read dP(j)
// and compute; dQ(j) comes last.  K_j is read by S(j) and by dQ(j); with the
// MMA order S(j+1), dP(j+1), dQ(j) the load of K(j+4) into the stage of K(j)
// has three tile groups of MMAs to land.

constexpr int Q_KST = 4;
constexpr int FEW_KEYS = 64;     // rows that see fewer get an exact Delta
enum {
    Q_QTM = 0,                   // Q tile landed
    Q_DOFULL = 1,                // dO rows in tensor memory (8 arrivals: the gradient warps)
    Q_KFULL = 2,                 // Q_KST stages
    Q_KEMPTY = 2 + Q_KST,        // Q_KST stages; commits after S(j) and after dQ(j)
    Q_VFULL = 2 + 2 * Q_KST,     // 2 stages
    Q_VEMPTY = 4 + 2 * Q_KST,    // 2 stages
    Q_SDONE = 6 + 2 * Q_KST,     // S(j) complete
    Q_PDONE = 7 + 2 * Q_KST,     // dP(j) complete
    Q_SFREE = 8 + 2 * Q_KST,     // S(j) read by the gradient warps (8 arrivals)
    Q_PFREE = 9 + 2 * Q_KST,     // dP(j) read (8 arrivals)
    Q_DS = 10 + 2 * Q_KST,       // dS(j) written (8 arrivals)
    Q_DSFREE = 11 + 2 * Q_KST,   // dQ(j) complete: the dS columns may be rewritten
    Q_FIN = 12 + 2 * Q_KST,
    Q_DRAIN = 13 + 2 * Q_KST,    // one commit per issuer (2)
    Q_QEMPTY = 14 + 2 * Q_KST,   // a unit's S MMAs complete: the Q tile may be reloaded
    Q_DELTA = 15 + 2 * Q_KST,    // WIN: shares of an exact Delta written (8 arrivals)
    Q_NBAR = 16 + 2 * Q_KST
};

template <int D>
struct DqCfg {
    static constexpr int TB = Tile<D>::BYTES;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = TB;                    // Q_KST stages
    static constexpr int OFF_V = (1 + Q_KST) * TB;      // 2 stages
    static constexpr int OFF_BAR = (3 + Q_KST) * TB;
    static constexpr int OFF_MISC = OFF_BAR + 8 * Q_NBAR;
    static constexpr int OFF_FIX = OFF_MISC + 16;       // WIN: FixList
    static constexpr int OFF_DELTA = OFF_FIX + ((int)sizeof(FixList) + 15) / 16 * 16;   // WIN: [2][2][T] fp32
    static constexpr int NEED = OFF_DELTA + 4 * T * 4;
    static constexpr int SMEM = NEED > 120 * 1024 ? NEED : 120 * 1024;
    static_assert(SMEM <= 232448, "dQ kernel shared memory");
    static constexpr uint32_t TM_S = 0, TM_P = 128, TM_DQ = 256, TM_DS = 256 + D, TM_DO = 320 + D;
    static_assert(TM_DO + D / 2 <= 512, "dQ kernel tensor memory");
};

// stage index and phase parity of a ring of NS buffers, advanced once per use
template <int NS>
struct Ring {
    int st = 0, ph = 0;
    __device__ __forceinline__ void next()
    {
        if (++st == NS) {
            st = 0;
            ph ^= 1;
        }
    }
};

struct BwdArgs {
    int B, Hq, Hkv, S, D, N, causal, layout;
    float scale;
    int upc;            // query units (128 rows) per chunk
    int tpc;            // key tiles per chunk
    unsigned *err;
    uint64_t limit_ns;   // pipeline waits
    uint64_t drain_ns;   // waits that drain copies and MMAs before exit
    int Sk;              // windowed attention: keys (S counts query rows)
    Window win;          // windowed attention
    SinkPlan sp;
    float *part;         // the sinks' partial gradients (window_sinks.cuh)
    float *delta;        // WIN: Delta, written by the dQ kernel
    int n_units;         // windowed attention: units of the launch
    FastDiv by_tiles, by_heads, by_group;   // of its numbering: tiles, heads (query or kv), Hq / Hkv
    FixArgs fix;         // windowed attention
};

// WIN: windowed attention with sinks, the walks of WinIter and WinQIter.  The dQ
// kernel's packed first tile has boxes of its own, as the forward's.  Units are short
// (about 10 tiles for a window of 1024), so a block takes several in turn: barrier phases
// run on across them (without WIN every unit loop runs once and the running counts are
// the unit's own), the next unit's loads and first products go out beside the current
// one's last steps, and its set-up is paid once (16384 rows, 16 heads, window 1024: dQ 241 us
// with a block a unit, 190 so).
struct PackMaps {
    CUtensorMap k_sinks, k_rest, v_sinks, v_rest;
};
struct NoMaps {
};

// WIN: the block's u-th unit; false: it has no more.
__device__ __forceinline__ bool window_q_unit(const BwdArgs &a, int u, Unit &w)
{
    const int64_t item = blockIdx.x + (int64_t)u * gridDim.x;
    if (item >= a.n_units) return false;
    const unsigned r = a.by_tiles.div((unsigned)item), t = (unsigned)item - r * (unsigned)a.upc;
    w.b = (int)a.by_heads.div(r);
    w.h = (int)r - w.b * a.Hq;
    w.r = 0;
    w.q0 = (int)t * T;
    w.cend = a.S;
    w.qmax = (w.q0 + T < a.S ? w.q0 + T : a.S) - 1;
    return true;
}

// WIN: the noted rows again (window_fix.cuh), by the gradient warps.
template <int D>
__device__ __noinline__ void dq_fix(const FixList &list, const BwdArgs &a, __nv_bfloat16 *dq)
{
    const int warp = (threadIdx.x >> 5) - 4;
    auto task = [&](const Unit &w, int quarter) {
        for (int r = 0; r < 32; ++r) {
            const int i = w.q0 + 32 * quarter + r;
            if (i < w.cend) fix::dq_row<D>(a.fix, w.b, w.h, i, dq);
        }
    };
    Unit w;
    if (list.count <= FixList::CAP) {
        for (int e = warp; e < list.count; e += 8)
            if (window_q_unit(a, list.entry[e] >> 3, w)) task(w, list.entry[e] & 3);
    } else {
        for (int u = 0; window_q_unit(a, u, w); ++u)
            if (warp < 4) task(w, warp);
    }
}

template <int D, bool WIN>
__global__ void __launch_bounds__(NTHREADS, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                  const __grid_constant__ BwdArgs a, const float *__restrict__ lse,
                  const float *__restrict__ delta, __nv_bfloat16 *__restrict__ dq,
                  const __nv_bfloat16 *__restrict__ dout,
                  const __grid_constant__ std::conditional_t<WIN, PackMaps, NoMaps> pm)
{
    using C = DqCfg<D>;
    using Walk = std::conditional_t<WIN, WinIter<T>, KvIter<T>>;
    constexpr int TB = C::TB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {   // the 128B-swizzled tiles need 1 KB alignment
        if (threadIdx.x == 0) atomicCAS(a.err, 0u, ERRW_SMEM_ALIGN);
        return;
    }
    const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K,
                   sV = base + C::OFF_V, bar0 = base + C::OFF_BAR;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem_raw + C::OFF_MISC + 4);
    FixList *fixes = reinterpret_cast<FixList *>(smem_raw + C::OFF_FIX);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Geom g = make_geom(a.S, a.N, a.layout, a.causal);
    struct Item {
        Unit w;
        int kvh, n;      // kv head, key tiles
        bool twice;      // WIN: the tiles pass twice, first for Delta
        __device__ __forceinline__ int passes() const { return WIN && twice ? 2 * n : n; }   // tiles, both times
    };
    // the block's it-th unit; false: it has no more
    auto unit_of = [&](int it, Item &x) -> bool {
        if constexpr (WIN) {
            if (!window_q_unit(a, it, x.w)) return false;
            x.kvh = (int)a.by_group.div((unsigned)x.w.h);
            const int p0 = x.w.q0 + a.win.off;
            x.n = WinIter<T>::count(a.win, p0, x.w.qmax + a.win.off);
            const int behind = p0 + 1 - a.win.window;   // keys behind the first row's window
            x.twice = (behind < 0 ? p0 + 1 : a.win.window + (behind < a.win.sinks ? behind : a.win.sinks)) < FEW_KEYS;
        } else {
            if (it > 0) return false;
            x.twice = false;
            x.w = decode_unit_grouped(g, a.B, a.Hq, a.upc, T, blockIdx.x);
            x.kvh = x.w.h / (a.Hq / a.Hkv);
            x.n = KvIter<T>::count(g, x.w.r, x.w.qmax);
        }
        return true;
    };
    auto start_walk = [&](Walk &it, const Unit &w) {
        if constexpr (WIN) it.begin(a.win, w.q0 + a.win.off, w.qmax + a.win.off);
        else it.begin(g, w.r, w.qmax);
    };
    // extents of the tensor maps' (rank, row) dimensions, for the debug-bounds build
    const int map_r = striped(g) ? g.N : 1, map_rows = a.S / map_r;
    // a tile of K or V into shared memory
    auto load_tile = [&](const Item &x, const Walk &it, uint32_t dst, const CUtensorMap *map, const CUtensorMap *sinks,
                         const CUtensorMap *rest, uint32_t bar, uint64_t policy) {
        if constexpr (WIN) {
            if (it.packed()) {
                for (int bx = 0; bx < D / 64; ++bx) {
                    tma_load5(dst + bx * 16384, sinks, bar, bx * 64, x.kvh, 0, 0, x.w.b, policy);
                    tma_load5(dst + bx * 16384 + it.pk * 128, rest, bar, bx * 64, x.kvh, 0,
                              dbg_coord(a.err, it.start() + it.pk, a.Sk), x.w.b, policy);
                }
                return;
            }
            const int row = dbg_coord(a.err, it.start(), a.Sk);
            for (int bx = 0; bx < D / 64; ++bx)
                tma_load5(dst + bx * 16384, map, bar, bx * 64, x.kvh, 0, row, x.w.b, policy);
        } else {
            const int mr = dbg_coord(a.err, it.mrank(), map_r), mw = dbg_coord(a.err, it.mrow(), map_rows);
            for (int bx = 0; bx < D / 64; ++bx)
                tma_load5(dst + bx * 16384, map, bar, bx * 64, x.kvh, mr, mw, x.w.b, policy);
        }
    };
    const CUtensorMap *pks = nullptr, *pkr = nullptr, *pvs = nullptr, *pvr = nullptr;
    if constexpr (WIN) pks = &pm.k_sinks, pkr = &pm.k_rest, pvs = &pm.v_sinks, pvr = &pm.v_rest;

    if (threadIdx.x == 0) {
        mbar_init(BAR(Q_QTM), 1);
        mbar_init(BAR(Q_DOFULL), 8);
        for (int i = 0; i < Q_KST; ++i) {
            mbar_init(BAR(Q_KFULL + i), 1);
            mbar_init(BAR(Q_KEMPTY + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(Q_VFULL + i), 1);
            mbar_init(BAR(Q_VEMPTY + i), 1);
        }
        mbar_init(BAR(Q_SDONE), 1);
        mbar_init(BAR(Q_PDONE), 1);
        mbar_init(BAR(Q_SFREE), 8);
        mbar_init(BAR(Q_PFREE), 8);
        mbar_init(BAR(Q_DS), 8);
        mbar_init(BAR(Q_DSFREE), 1);
        mbar_init(BAR(Q_FIN), 1);
        mbar_init(BAR(Q_DRAIN), 2);
        mbar_init(BAR(Q_QEMPTY), 1);
        mbar_init(BAR(Q_DELTA), 8);
        *abort_flag = 0;
        if constexpr (WIN) fixes->count = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{a.err, abort_flag, a.limit_ns};

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CTRL));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------------ K producer
            const uint64_t pol_kv = policy_evict_last();
            int nk = 0;
            Ring<Q_KST> kr;
            Item x;
            bool ok = true;
            for (int u = 0; ok && unit_of(u, x); ++u) {
                Walk it;
                start_walk(it, x.w);
                for (int j = 0; j < x.passes(); ++j, it.next(), kr.next()) {
                    if (WIN && x.twice && j == x.n) start_walk(it, x.w);
                    if (nk >= Q_KST && !wait1(BAR(Q_KEMPTY + kr.st), kr.ph ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(BAR(Q_KFULL + kr.st), TB);
                    load_tile(x, it, sK + kr.st * TB, &tmK, pks, pkr, BAR(Q_KFULL + kr.st), pol_kv);
                    ++nk;
                }
            }
            {
                // wait (bounded) for the copies still in flight before the block
                // exits: always, since a consumer may give up after the last copy
                // was issued (after a normal run these phases are complete)
                volatile int no_abort = 0;
                WaitCtl dc{a.err, &no_abort, a.drain_ns};
                for (int j = nk > Q_KST ? nk - Q_KST : 0; j < nk; ++j)
                    wait1(BAR(Q_KFULL + j % Q_KST), (j / Q_KST) & 1, dc);
            }
        } else if (warp == 3 && lane == 0) {
            // ------------------------------------------------------------ dO and V producer
            const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
            int nv = 0, nq = 0;
            Item x;
            bool ok = true;
            for (int u = 0; ok && unit_of(u, x); ++u) {
                if (u > 0 && !wait1(BAR(Q_QEMPTY), (u - 1) & 1, wc)) break;
                const int qmr = WIN ? 0 : dbg_coord(a.err, slot_mrank(g, x.w.q0), map_r);
                const int qmw = WIN ? dbg_coord(a.err, x.w.q0, a.S) : dbg_coord(a.err, slot_mrow(g, x.w.q0), map_rows);
                mbar_arrive_expect_tx(BAR(Q_QTM), TB);
                for (int bx = 0; bx < D / 64; ++bx)
                    tma_load5(sQ + bx * 16384, &tmQ, BAR(Q_QTM), bx * 64, x.w.h, qmr, qmw, x.w.b, pol_q);
                ++nq;
                Walk it;
                start_walk(it, x.w);
                for (int j = 0; j < x.passes(); ++j, it.next()) {
                    if (WIN && x.twice && j == x.n) start_walk(it, x.w);
                    const int sv = nv & 1;
                    if (nv >= 2 && !wait1(BAR(Q_VEMPTY + sv), ((nv >> 1) - 1) & 1, wc)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(BAR(Q_VFULL + sv), TB);
                    load_tile(x, it, sV + sv * TB, &tmV, pvs, pvr, BAR(Q_VFULL + sv), pol_kv);
                    ++nv;
                }
            }
            {
                volatile int no_abort = 0;
                WaitCtl dc{a.err, &no_abort, a.drain_ns};
                if (nq > 0) wait1(BAR(Q_QTM), (nq - 1) & 1, dc);
                for (int j = nv > 2 ? nv - 2 : 0; j < nv; ++j) wait1(BAR(Q_VFULL + (j & 1)), (j >> 1) & 1, dc);
            }
        } else if (warp == 1 || warp == 2) {
            // ------------------------------------------------------------ MMA issuers
            // warp 1: S = Q K^T (A = Q from tensor memory) and dP = dO V^T;
            // warp 2: dQ += dS K.  Each warp runs converged (warp-collective
            // waits), so its operands stay warp-uniform, and one elected lane
            // issues the MMAs and their commits.
            constexpr uint32_t idSP = idesc_bf16(128, T, false);     // K-major A and B
            constexpr uint32_t idDQ = idesc_bf16(128, D, true);      // B = K MN-major
            const uint32_t tS = tmem + C::TM_S, tP = tmem + C::TM_P, tDQ = tmem + C::TM_DQ,
                           tDS = tmem + C::TM_DS, tDO = tmem + C::TM_DO;
            const bool leader = elect_one();
            bool ok = true;
            if (warp == 1) {
                const uint64_t dQd = sdesc(sQ, 16, 1024);
                const uint64_t dK0 = sdesc(sK, 16, 1024), dV0 = sdesc(sV, 16, 1024);
                Ring<Q_KST> kr;
                Item x;
                int nt = 0;
                for (int u = 0; ok && unit_of(u, x); ++u) {
                    if (!waitw(BAR(Q_QTM), u & 1, wc)) break;
                    const int n = x.passes();
                    for (int j = 0; j < n; ++j, ++nt, kr.next()) {
                        const int sv = nt & 1;
                        if ((nt > 0 && !waitw(BAR(Q_SFREE), (nt - 1) & 1, wc)) ||
                            !waitw(BAR(Q_KFULL + kr.st), kr.ph, wc)) {
                            ok = false;
                            break;
                        }
                        const uint64_t dK = dK0 + (uint64_t)(kr.st * (TB >> 4));
                        if (leader) {
                            tc_fence_after();
                            ss_seq<0, D, 16384>(tS, dQd, dK, idSP);
                            mma_commit(BAR(Q_SDONE));
                            mma_commit(BAR(Q_KEMPTY + kr.st));
                            if (WIN && j + 1 == n) mma_commit(BAR(Q_QEMPTY));
                        }
                        __syncwarp();
                        if ((nt > 0 && !waitw(BAR(Q_PFREE), (nt - 1) & 1, wc)) ||
                            (j == 0 && !waitw(BAR(Q_DOFULL), u & 1, wc)) || !waitw(BAR(Q_VFULL + sv), (nt >> 1) & 1, wc)) {
                            ok = false;
                            break;
                        }
                        const uint64_t dV = dV0 + (uint64_t)(sv * (TB >> 4));
                        if (leader) {
                            tc_fence_after();
                            ts_k_seq<0, D>(tP, tDO, dV, idSP);   // A = dO from tensor memory
                            mma_commit(BAR(Q_PDONE));
                            mma_commit(BAR(Q_VEMPTY + sv));
                        }
                        __syncwarp();
                    }
                }
            } else {
                const uint64_t dKmn0 = sdesc(sK, 16384, 1024);
                Ring<Q_KST> kr;
                Item x;
                int nt = 0;
                for (int u = 0; ok && unit_of(u, x); ++u) {
                    const int n = x.passes(), j0 = n - x.n;   // the tiles from j0 on have a dS
                    for (int j = 0; j < n; ++j, ++nt, kr.next()) {
                        // dS(nt) written: the gradient warps have also read the previous
                        // unit's dQ, which this unit's first product overwrites
                        if (!waitw(BAR(Q_DS), nt & 1, wc) || !waitw(BAR(Q_KFULL + kr.st), kr.ph, wc)) {
                            ok = false;
                            break;
                        }
                        const uint64_t dK = dKmn0 + (uint64_t)(kr.st * (TB >> 4));
                        const uint32_t acc0 = j > j0 ? 1u : 0u;
                        if (leader) {
                            tc_fence_after();
                            if (j >= j0) ts_mn_seq<0, T / 16, 0>(tDQ, tDS, dK, idDQ, acc0);
                            mma_commit(BAR(Q_KEMPTY + kr.st));
                            mma_commit(BAR(Q_DSFREE));
                            if (j + 1 == n) mma_commit(BAR(Q_FIN));
                        }
                        __syncwarp();
                    }
                }
            }
            if (leader) mma_commit(BAR(Q_DRAIN));
            __syncwarp();
            volatile int no_abort = 0;
            WaitCtl dc{a.err, &no_abort, a.drain_ns};
            waitw(BAR(Q_DRAIN), 0, dc);
        }
        __syncwarp();
        tc_fence_before();
        asm volatile("barrier.sync 1, %0;" ::"n"(NTHREADS) : "memory");
        if (warp == 0) {
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        }
        return;
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_GRAD));
        // ------------------------------------------------------------ dS = P (dP - Delta)
        const int half = (warp - 4) >> 2;             // columns [64*half, 64*half+64)
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + C::TM_S + 64u * half;
        const uint32_t tP = tmem + lane_off + C::TM_P + 64u * half;
        const uint32_t tDQ = tmem + lane_off + C::TM_DQ;
        const uint32_t tDS = tmem + lane_off + C::TM_DS + 32u * half;
        const float sl2 = a.scale * LOG2E;
        // This thread's row of a unit: its statistics, and its half of the row's dO, as D/4
        // bf16 pairs, into the A operand of dP = dO V^T (rows past the unit's chunk are zero;
        // their results are never stored).  The dO columns are free once dP of the previous
        // unit's last tile has been read.
        struct Row {
            int qpos, qp;      // slot, global position
            bool valid;
            float lse2, dlt;
        };
        // WIN: Delta = rowsum(dO out) is made here, while the tensor cores finish the unit before,
        // and written for dK / dV: 201 us for both (16384 rows, 16 heads, window 1024), where a
        // kernel of its own took 30 and this one 190.  Rows come in chunks that cover whole
        // sectors, from L2, where the unit before had them sent (every lane its own row, from
        // memory: 244).  Each half leaves its share in shared memory, by the unit's parity;
        // Q_DOFULL tells of both.
        // out has been rounded to bf16, which Delta takes over: an error of 2^-9 sqrt(sum P^2) of
        // dQ and dK, as large as their own rounding where a row sees few keys.  Units with such
        // rows (Item::twice) pass their tiles, two at most, twice, the first time for Delta =
        // sum_j P dP in fp32.  (Window of 2: dQ off by 0.0024 of its norm where it was 0.0038, the
        // rounding of the result alone is 0.0017; windows below 64 take 185 us a step of 8192 rows
        // and 16 heads where they took 162, longer ones 1 to 3 us more.)
        float *shares = reinterpret_cast<float *>(smem_raw + C::OFF_DELTA);
        const bool rows32 = WIN && ((reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(a.fix.out)) & 31) == 0;
        auto load_row = [&](const Unit &w, int u) -> Row {
            Row r;
            r.qpos = w.q0 + row;
            r.valid = r.qpos < w.cend;
            if constexpr (WIN) r.qp = dbg_coord(a.err, r.valid ? r.qpos : 0, a.S);
            else r.qp = dbg_coord(a.err, r.valid ? slot_pos(g, r.qpos) : 0, a.S);
            r.lse2 = r.dlt = 0.f;
            uint32_t dv4[D / 4];
            if (r.valid) {
                r.lse2 = lse[((int64_t)w.b * a.Hq + w.h) * a.S + r.qp] * LOG2E;
                if constexpr (!WIN) r.dlt = delta[((int64_t)w.b * a.Hq + w.h) * a.S + r.qp];
            }
            if constexpr (WIN) {
                // lane c of a group of G loads chunk c, 32 bytes, of the group's pieces in turn
                constexpr int G = D / 32;
                const int c = lane & (G - 1), gb = lane & ~(G - 1);
                const int64_t at = (((int64_t)w.b * a.S + w.q0 + quarter * 32 + gb) * a.Hq + w.h) * D + (D / 2) * half + 16 * c;
                uint32_t ld[G][8], lo[G][8];
#pragma unroll
                for (int m = 0; m < G; ++m) {
                    const bool there = w.q0 + quarter * 32 + gb + m < w.cend;
                    load_chunk(dout + at + (int64_t)m * a.Hq * D, there, rows32, ld[m]);
                    load_chunk(a.fix.out + at + (int64_t)m * a.Hq * D, there, rows32, lo[m]);
                }
#pragma unroll
                for (int m = 0; m < G; ++m) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s0 = fmaf(__uint_as_float(lo[m][e] << 16), __uint_as_float(ld[m][e] << 16), s0);
                        s1 = fmaf(__uint_as_float(lo[m][e] & 0xffff0000u), __uint_as_float(ld[m][e] & 0xffff0000u), s1);
                    }
                    s0 += s1;
#pragma unroll
                    for (int o = 1; o < G; o <<= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                    if (c == m) r.dlt = s0;
                }
                chunks_to_pieces(ld, dv4, c);
            } else if (r.valid) {
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    dout + (((int64_t)w.b * a.S + r.qp) * a.Hq + w.h) * D + (D / 2) * half);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint4 v = src[i];
                    dv4[4 * i] = v.x;
                    dv4[4 * i + 1] = v.y;
                    dv4[4 * i + 2] = v.z;
                    dv4[4 * i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) dv4[i] = 0u;
            }
            const uint32_t tDO = tmem + lane_off + C::TM_DO + (uint32_t)(D / 4) * half;
            if constexpr (D == 128)
                tmem_st_x32(tDO, dv4);
            else
                tmem_st_x16(tDO, dv4);
            if constexpr (WIN) shares[((u & 1) * 2 + half) * T + row] = r.dlt;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(Q_DOFULL));
            return r;
        };
        bool ok = true;
        int nt = 0, nd = 0;                            // tiles, units with an exact Delta so far
        Item xn;
        bool have = unit_of(0, xn);
        Row rn{};
        if (have) rn = load_row(xn.w, 0);
        for (int u = 0; ok && have; ++u) {
            const Item x = xn;
            const Unit &w = x.w;
            const Row rw = rn;
            const int qpos = rw.qpos, qp = rw.qp;
            const bool valid = rw.valid;
            float sum = 0.f;                           // of P dP, the first time
            const float lse2 = rw.lse2;
            float dlt = rw.dlt;
            if constexpr (WIN) {
                if (!waitw(BAR(Q_DOFULL), u & 1, wc)) break;
                if (!x.twice) {
                    const float *share = shares + (u & 1) * 2 * T + row;
                    dlt = share[0] + share[T];
                    if (valid && half == 0) a.delta[((int64_t)w.b * a.Hq + w.h) * a.S + qp] = dlt;
                }
                Item y;
                if (unit_of(u + 1, y) && y.w.q0 + row < a.S) {   // the next unit's rows, on their way to L2
                    const int64_t at = (((int64_t)y.w.b * a.S + y.w.q0 + row) * a.Hq + y.w.h) * D + (D / 2) * half;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(dout + at));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.fix.out + at));
                }
            }
            Walk it;
            start_walk(it, w);
            // one tile; FIRST: for Delta.  False: a wait ran out.
            auto tile = [&](auto first) -> bool {
                constexpr bool FIRST = decltype(first)::value;
                const int ks = it.start(), kl = it.len();
                int lim = kl;                              // visible columns [0, lim) of the tile
                uint32_t see0 = 0xffffffffu, see1 = 0xffffffffu;   // WIN: visible columns, 32 each
                bool all = false;
                if constexpr (WIN) {
                    const int p0 = w.q0 + a.win.off, p = qpos + a.win.off;
                    all = it.full(a.win, p0, w.qmax + a.win.off);
                    if (!all) {
                        const int hi = (p - ks + 1 < kl ? p - ks + 1 : kl) - 64 * half;
                        const int lo = it.window_col(a.win, p) - 64 * half, sc = it.sink_cols() - 64 * half;
                        see0 = visible_bits(0, hi, lo, sc);
                        see1 = visible_bits(32, hi, lo, sc);
                    }
                } else {
                    if (a.causal) {
                        const int c = qpos - ks + 1 + it.shift;
                        lim = c < lim ? c : lim;
                    }
                }
                lim -= 64 * half;                          // in this half's local columns
                if (!waitw(BAR(Q_SDONE), nt & 1, wc)) return false;
                tc_fence_after();
                uint32_t sr[64];
                tmem_ld_x64(tS, sr);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(Q_SFREE));   // S(j+1) may be issued
                // P = exp2(S sl2 - lse2); the per-element mask only where some row of
                // the warp does not see the whole half tile
                const bool full = WIN ? all : __all_sync(0xffffffffu, lim >= 64);
                float p[64];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    ffma2(p[e], p[e + 1], __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]), sl2, -lse2);
                    p[e] = ex2(p[e]);
                    p[e + 1] = ex2(p[e + 1]);
                }
                if (!full) {
                    if constexpr (WIN) {
                        // runs of 32 columns that the whole warp sees are left alone
                        if (!__all_sync(0xffffffffu, see0 == 0xffffffffu)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) p[e] = see0 & (1u << e) ? p[e] : 0.f;
                        }
                        if (!__all_sync(0xffffffffu, see1 == 0xffffffffu)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) p[32 + e] = see1 & (1u << e) ? p[32 + e] : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 64; ++e) p[e] = e < lim ? p[e] : 0.f;
                    }
                }
                if (!waitw(BAR(Q_PDONE), nt & 1, wc)) return false;
                tc_fence_after();
                uint32_t pr[64];
                tmem_ld_x64(tP, pr);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(Q_PFREE));   // dP(j+1) may be issued
                if constexpr (FIRST) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)           // (dP of what the row does not see may be NaN)
                        sum = p[e] == 0.f ? sum : fmaf(p[e], __uint_as_float(pr[e]), sum);
                    if (nt > 0 && !waitw(BAR(Q_DSFREE), (nt - 1) & 1, wc)) return false;
                    if (lane == 0) mbar_arrive(BAR(Q_DS));
                    return true;
                }
                // dS = P (dP - Delta)
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float t0, t1;
                    fadd2v(t0, t1, __uint_as_float(pr[2 * e]), __uint_as_float(pr[2 * e + 1]), -dlt, -dlt);
                    fmul2v(t0, t1, t0, t1, p[2 * e], p[2 * e + 1]);
                    pk[e] = pack_bf16(t0, t1);
                }
                // dS(j) may be written once dQ(j-1) has read dS(j-1)
                if (nt > 0 && !waitw(BAR(Q_DSFREE), (nt - 1) & 1, wc)) return false;
                tc_fence_after();
                tmem_st_x32(tDS, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(Q_DS));
                return true;
            };
            if constexpr (WIN) {
                if (x.twice) {
                    for (int j = 0; ok && j < x.n; ++j, ++nt, it.next()) ok = tile(std::true_type{});
                    if (!ok) break;
                    start_walk(it, w);
                    float *share = shares + (u & 1) * 2 * T + row;
                    share[half * T] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(Q_DELTA));
                    if (!waitw(BAR(Q_DELTA), nd & 1, wc)) break;
                    ++nd;
                    dlt = share[0] + share[T];
                    if (valid && half == 0) a.delta[((int64_t)w.b * a.Hq + w.h) * a.S + qp] = dlt;
                }
            }
            for (int j = 0; ok && j < x.n; ++j, ++nt, it.next()) ok = tile(std::false_type{});
            // the next unit's rows first: its S and dP run beside this unit's epilogue
            have = ok && unit_of(u + 1, xn);
            if (have) rn = load_row(xn.w, u + 1);
            if (ok && waitw(BAR(Q_FIN), u & 1, wc)) {
                tc_fence_after();
                // each half writes D/2 columns of dQ = scale * acc
                constexpr int HD = D / 2;
                const bool a32 = (reinterpret_cast<uintptr_t>(dq) & 31) == 0;
                float odd = 0.f;
                __nv_bfloat16 *orow = dq + (((int64_t)w.b * a.S + qp) * a.Hq + w.h) * D + HD * half;
#pragma unroll (WIN ? 1 : HD / 32)
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_x32(tDQ + HD * half + 32u * c, o);
                    if constexpr (WIN) {
                        odd += odd_columns(o);
                        if (a32) {
                            put_row_piece(orow + 32 * c, valid, o, a.scale, lane);
                            continue;
                        }
                    }
                    if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(orow + 32 * c);
#pragma unroll
                        for (int v4 = 0; v4 < 4; ++v4) {
                            uint4 pkt;
                            pkt.x = pack_bf16(__uint_as_float(o[8 * v4 + 0]) * a.scale, __uint_as_float(o[8 * v4 + 1]) * a.scale);
                            pkt.y = pack_bf16(__uint_as_float(o[8 * v4 + 2]) * a.scale, __uint_as_float(o[8 * v4 + 3]) * a.scale);
                            pkt.z = pack_bf16(__uint_as_float(o[8 * v4 + 4]) * a.scale, __uint_as_float(o[8 * v4 + 5]) * a.scale);
                            pkt.w = pack_bf16(__uint_as_float(o[8 * v4 + 6]) * a.scale, __uint_as_float(o[8 * v4 + 7]) * a.scale);
                            dst[v4] = pkt;
                        }
                    }
                }
                if constexpr (WIN) {
                    if (__any_sync(0xffffffffu, valid && !(odd == 0.f)) && lane == 0) fixes->note(u, quarter);
                }
            }
        }
        __syncwarp();
        tc_fence_before();
        asm volatile("barrier.sync 1, %0;" ::"n"(NTHREADS) : "memory");
        if constexpr (WIN) {
            if (fixes->count > 0) dq_fix<D>(*fixes, a, dq);
        }
        return;
    }
#undef BAR
}

// ----------------------------------------------------------------------------- dK, dV
//
// Key-stationary, in half tiles of 64 queries: for each query tile the block
// visits (QIter order), two half steps s.  Per half step: S^T = K Q_s^T and
// dP^T = V dO_s^T (M=128 keys, N=64) into tensor-memory buffer s%2; gradient
// warpgroup s%2 turns them into P^T and dS^T (bf16 pairs, written over the
// first half of the columns it read); then dV += P^T dO_s and dK += dS^T Q_s
// (N=D, K=64).  With two buffers and one warpgroup per buffer, the MMAs of
// step s+1 run while warpgroup s%2 works on step s.  S^T and dP^T have
// barriers of their own: S^T(s+2) is issued into buffer s%2 once dV(s) has
// read P^T(s) out of the S^T columns, dP^T(s+2) once dK(s) has read dS^T(s)
// out of the dP^T columns (commit barriers, since the MMA groups come from
// different issuing warps), and the gradient warps turn S^T into P^T before
// they wait for dP^T.  A buffer's serial chain is then P^T -> dV -> S^T of
// the step after next, without the dS^T and dK stages.
// Each gradient thread handles all 64 columns of its steps, so it moves them
// with two 64-column tensor-memory loads and two 32-column stores.
//
// Tensor memory (columns): buffer x at 128x: S^T [0,64), dP^T [64,128);
// dV [256, 256+D), dK [256+D, 256+2D).  Shared memory: K and V (128 rows),
// K_QST half stages of (Q_s, dO_s) 64-row tiles, and their lse / Delta.

constexpr int K_QST = 5;
enum {
    K_KVFULL = 0,
    K_QFULL = 1,                  // K_QST half stages
    K_QEMPTY = 1 + K_QST,         // K_QST half stages
    K_S = 1 + 2 * K_QST,          // 2 buffers: S^T complete
    K_PW = 3 + 2 * K_QST,         // 2 buffers: P^T written (4 arrivals: one warpgroup)
    K_SFREE = 5 + 2 * K_QST,      // 2 buffers: dV(s) complete, the S^T columns may be rewritten
    K_FIN = 7 + 2 * K_QST,
    K_DRAIN = 8 + 2 * K_QST,      // one commit per issuing warp (3)
    K_DSW = 9 + 2 * K_QST,        // 2 buffers: dS^T written (4 arrivals)
    K_DP = 11 + 2 * K_QST,        // 2 buffers: dP^T complete
    K_DPFREE = 13 + 2 * K_QST,    // 2 buffers: dK(s) complete, the dP^T columns may be rewritten
    K_KVEMPTY = 15 + 2 * K_QST,   // a unit's S^T and dP^T MMAs complete (2): K and V may be reloaded
    K_ACC = 16 + 2 * K_QST,       // a unit's dK read by its warpgroup (4 arrivals)
    K_FINV = 17 + 2 * K_QST,      // WIN: a unit's dV complete (its dK: K_FIN)
    K_NBAR = 18 + 2 * K_QST
};

template <int D>
struct DkvCfg {
    static constexpr int TB = Tile<D>::BYTES;            // 128 rows
    static constexpr int HB = TB / 2;                    // 64 rows
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = TB;
    static constexpr int OFF_Q = 2 * TB;                 // K_QST stages of (Q_s, dO_s)
    static constexpr int STAGE = 2 * HB;
    static constexpr int OFF_STAT = OFF_Q + K_QST * STAGE;   // K_QST x (lse2[64], delta[64]) fp32
    static constexpr int OFF_BAR = OFF_STAT + K_QST * 2 * 64 * 4;
    static constexpr int OFF_MISC = OFF_BAR + 8 * K_NBAR;
    static constexpr int OFF_FIX = OFF_MISC + 16;            // WIN: FixList
    static constexpr int NEED = OFF_FIX + (int)sizeof(FixList);
    static constexpr int SMEM = NEED > 120 * 1024 ? NEED : 120 * 1024;
    static_assert(SMEM <= 232448, "dK/dV kernel shared memory");
    static constexpr uint32_t TM_DV = 256, TM_DK = 256 + D;
    static_assert(TM_DK + D <= 512, "dK/dV kernel tensor memory");
};

// Where key row j's gradient goes: dK's (k) or dV's row, or a sink's partial.
template <int D>
__device__ __forceinline__ float *partial_row(const BwdArgs &a, int b, int g, int piece, int j, bool k)
{
    if (a.sp.pieces == 0 || j >= a.win.sinks) return nullptr;
    return a.part + (((int64_t)b * a.Hkv + g) * window_part_rows(a.win, a.sp) + ((int64_t)piece * 2 + (k ? 0 : 1)) * a.win.sinks + j) * D;
}

// WIN: the block's u-th unit and its piece (0: a window unit, else 1 + the piece of a tile of
// sinks); false: it has no more.
__device__ __forceinline__ bool window_kv_unit(const BwdArgs &a, int u, KvUnit &w, int &piece)
{
    const int64_t item = blockIdx.x + (int64_t)u * gridDim.x;
    if (item >= a.n_units) return false;
    const int windows = a.tpc * a.B * a.Hkv;
    unsigned t, r;
    if (item < windows) {
        piece = 0;
        r = a.by_tiles.div((unsigned)item);
        t = (unsigned)item - r * (unsigned)a.tpc;
    } else {
        const unsigned y = (unsigned)(item - windows), z = y / (unsigned)a.sp.pieces;
        piece = 1 + (int)(y - z * (unsigned)a.sp.pieces);
        r = z / (unsigned)a.sp.tiles;
        t = z - r * (unsigned)a.sp.tiles;
    }
    w.b = (int)a.by_heads.div(r);
    w.g = (int)r - w.b * a.Hkv;
    w.src = 0;
    w.ks = (int)t * T;
    w.kcend = a.Sk;
    w.kl = a.Sk - w.ks < T ? a.Sk - w.ks : T;
    return true;
}

// WIN: the noted rows again (window_fix.cuh), by the gradient warps: warps 0 to 3 of a unit
// wrote dV, 4 to 7 dK.
template <int D>
__device__ __noinline__ void dkdv_fix(const FixList &list, const BwdArgs &a, __nv_bfloat16 *dk, __nv_bfloat16 *dv)
{
    const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31, grp = a.Hq / a.Hkv;
    auto task = [&](const KvUnit &w, int piece, int which) {
        const bool k = which >= 4;
        for (int r = 0; r < 32; ++r) {
            const int row = 32 * (which & 3) + r, j = w.ks + row;
            if (row >= w.kl) return;
            float *prow = partial_row<D>(a, w.b, w.g, piece, j, k);
            if (!prow && piece != 0) continue;
            __nv_bfloat16 *brow = (k ? dk : dv) + (((int64_t)w.b * a.Sk + j) * a.Hkv + w.g) * D;
            fix::Piece<D> was{}, acc{};
            if (prow) {
#pragma unroll
                for (int e = 0; e < D / 32; ++e) was.x[e] = prow[2 * lane + 64 * (e >> 1) + (e & 1)];
            } else {
                was = fix::load<D>(brow, lane);
            }
            if (fix::finite(was)) continue;
            if (piece == 0) {
                const int i0 = j - a.win.off > 0 ? j - a.win.off : 0;
                const int64_t i1 = (int64_t)j - a.win.off + a.win.window;
                for (int h = 0; h < grp; ++h)
                    if (fix::key_rows<D>(a.fix, w.b, w.g * grp + h, j, i0, (int)(i1 < a.S ? i1 : a.S), k, was, acc)) break;
            } else {
                WinQIter<T> it;
                for (it.sinks(a.win, a.S, w.ks, w.g * grp, grp, piece - 1, a.sp.each); it.count() > 0; it.next()) {
                    const int64_t from = (int64_t)j + a.win.window - a.win.off;   // the first row behind the window
                    const int i0 = from > it.start() ? (from < a.S ? (int)from : a.S) : it.start();
                    if (fix::key_rows<D>(a.fix, w.b, it.head(), j, i0, it.start() + it.len(), k, was, acc)) break;
                }
            }
            acc = fix::mended(was, acc, 1.f);
            if (prow) {
#pragma unroll
                for (int e = 0; e < D / 32; ++e) prow[2 * lane + 64 * (e >> 1) + (e & 1)] = acc.x[e];
            } else {
                fix::store(brow, acc, lane);
            }
        }
    };
    KvUnit w;
    int piece = 0;
    if (list.count <= FixList::CAP) {
        for (int e = warp; e < list.count; e += 8)
            if (window_kv_unit(a, list.entry[e] >> 3, w, piece)) task(w, piece, list.entry[e] & 7);
    } else {
        for (int u = 0; window_kv_unit(a, u, w, piece); ++u) task(w, piece, warp);
    }
}

template <int D, bool WIN>
__global__ void __launch_bounds__(NTHREADS, 1)
    bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tmQh, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDOh,
                    const __grid_constant__ BwdArgs a, const float *__restrict__ lse, const float *__restrict__ delta,
                    __nv_bfloat16 *__restrict__ dk, __nv_bfloat16 *__restrict__ dv)
{
    using C = DkvCfg<D>;
    constexpr int TB = C::TB, HB = C::HB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {   // the 128B-swizzled tiles need 1 KB alignment
        if (threadIdx.x == 0) atomicCAS(a.err, 0u, ERRW_SMEM_ALIGN);
        return;
    }
    const uint32_t sK = base + C::OFF_K, sV = base + C::OFF_V, sQ = base + C::OFF_Q,
                   bar0 = base + C::OFF_BAR;
    float *stat = reinterpret_cast<float *>(smem_raw + C::OFF_STAT);   // [stage][lse2 | delta][64]
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem_raw + C::OFF_MISC + 4);
    FixList *fixes = reinterpret_cast<FixList *>(smem_raw + C::OFF_FIX);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = a.Hq / a.Hkv;
    const Geom g = make_geom(a.S, a.N, a.layout, a.causal);
    using Walk = std::conditional_t<WIN, WinQIter<T>, QIter<T>>;
    struct Item {
        KvUnit w;
        int piece;       // WIN: 0 a window unit, else 1 + the piece of a tile of sinks
        int ns;          // half steps
    };
    auto start_walk = [&](Walk &it, const Item &x) {
        if constexpr (!WIN) it.begin(g, x.w.src, x.w.ks, x.w.g * grp, grp);
        else if (x.piece == 0) it.window(a.win, a.S, x.w.ks, x.w.kl, x.w.g * grp, grp);
        else it.sinks(a.win, a.S, x.w.ks, x.w.g * grp, grp, x.piece - 1, a.sp.each);
    };
    // the block's it-th unit; false: it has no more
    auto unit_of = [&](int it, Item &x) -> bool {
        x.piece = 0;
        if constexpr (WIN) {
            if (!window_kv_unit(a, it, x.w, x.piece)) return false;
            Walk wk;
            start_walk(wk, x);
            x.ns = 2 * wk.count();
        } else {
            if (it > 0) return false;
            x.w = decode_kv_unit<T>(g, a.B, a.Hkv, a.tpc, blockIdx.x);
            x.ns = 2 * QIter<T>::count(g, x.w.src, x.w.ks, grp);
        }
        return true;
    };
    // extents of the tensor maps' (rank, row) dimensions, for the debug-bounds build
    const int map_r = striped(g) ? g.N : 1, map_rows = a.S / map_r;

    if (threadIdx.x == 0) {
        mbar_init(BAR(K_KVFULL), 1);
        for (int i = 0; i < K_QST; ++i) {
            mbar_init(BAR(K_QFULL + i), 1);
            mbar_init(BAR(K_QEMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(K_S + i), 1);
            mbar_init(BAR(K_DP + i), 1);
            mbar_init(BAR(K_PW + i), 4);
            mbar_init(BAR(K_DSW + i), 4);
            mbar_init(BAR(K_SFREE + i), 1);
            mbar_init(BAR(K_DPFREE + i), 1);
        }
        mbar_init(BAR(K_FIN), 1);
        mbar_init(BAR(K_FINV), 1);
        mbar_init(BAR(K_DRAIN), 3);
        mbar_init(BAR(K_KVEMPTY), 2);
        mbar_init(BAR(K_ACC), 4);
        *abort_flag = 0;
        if constexpr (WIN) fixes->count = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{a.err, abort_flag, a.limit_ns};

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CTRL));
        if (warp == 0) {
            // ------------------------------------------------------------ producer (whole warp)
            const uint64_t pol_kv = policy_evict_first(), pol_q = policy_evict_last();
            int issued = 0, nkv = 0;
            Ring<K_QST> qr;
            Item x;
            bool ok = true;
            // Per-row statistics of a half tile, fetched a half step ahead (waiting for them
            // at every step held back a unit's first loads by a memory latency each):
            // -lse in log2 units and -Delta of rows lane and lane + 32.
            float st_l[2], st_d[2];
            auto fetch_stats = [&](const Walk &it, int hs) {
                const int qa = it.start() + 64 * hs, ql = it.len() - 64 * hs;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int e = lane + 32 * i;
                    st_l[i] = st_d[i] = 0.f;
                    if (e < ql) {
                        const int pos = WIN ? qa + e : slot_pos(g, qa + e);
                        const int64_t off = ((int64_t)x.w.b * a.Hq + it.head()) * a.S + dbg_coord(a.err, pos, a.S);
                        st_l[i] = lse[off];
                        st_d[i] = delta[off];
                    }
                }
            };
            for (int u = 0; ok && unit_of(u, x); ++u) {
                Walk it;
                start_walk(it, x);
                if (x.ns > 0) fetch_stats(it, 0);
                if (u > 0 && !waitw(BAR(K_KVEMPTY), (u - 1) & 1, wc)) break;
                if (lane == 0) {
                    const int kmr = WIN ? 0 : dbg_coord(a.err, slot_mrank(g, x.w.ks), map_r);
                    const int kmw =
                        WIN ? dbg_coord(a.err, x.w.ks, a.Sk) : dbg_coord(a.err, slot_mrow(g, x.w.ks), map_rows);
                    mbar_arrive_expect_tx(BAR(K_KVFULL), 2 * TB);
                    for (int bx = 0; bx < D / 64; ++bx) {
                        tma_load5(sK + bx * 16384, &tmK, BAR(K_KVFULL), bx * 64, x.w.g, kmr, kmw, x.w.b, pol_kv);
                        tma_load5(sV + bx * 16384, &tmV, BAR(K_KVFULL), bx * 64, x.w.g, kmr, kmw, x.w.b, pol_kv);
                    }
                }
                ++nkv;
                for (int s = 0; s < x.ns; ++s, qr.next()) {
                    if (issued >= K_QST && !waitw(BAR(K_QEMPTY + qr.st), qr.ph ^ 1, wc)) {
                        ok = false;
                        break;
                    }
                    const int hs = s & 1, h = it.head();
                    // map coordinates; the second half-tile may start past the end of
                    // the map (a short last tile): the copy then reads the fill value
                    int qr_rank = 0, qr_row;
                    if constexpr (WIN) {
                        qr_row = dbg_coord(a.err, it.start(), a.S) + 64 * hs;
                    } else {
                        qr_rank = dbg_coord(a.err, it.mrank(), map_r);
                        qr_row = dbg_coord(a.err, it.mrow(), map_rows) + 64 * hs;
                    }
                    float *ls = stat + qr.st * 128, *dl = ls + 64;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ls[lane + 32 * i] = -st_l[i] * LOG2E;
                        dl[lane + 32 * i] = -st_d[i];
                    }
                    __syncwarp();
                    if (lane == 0) {
                        const uint32_t sq = sQ + qr.st * C::STAGE;
                        mbar_arrive_expect_tx(BAR(K_QFULL + qr.st), 2 * HB);
                        for (int bx = 0; bx < D / 64; ++bx) {
                            tma_load5(sq + bx * 8192, &tmQh, BAR(K_QFULL + qr.st), bx * 64, h, qr_rank,
                                      qr_row, x.w.b, pol_q);
                            tma_load5(sq + HB + bx * 8192, &tmDOh, BAR(K_QFULL + qr.st), bx * 64, h, qr_rank,
                                      qr_row, x.w.b, pol_q);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (hs) it.next();
                    if (s + 1 < x.ns) fetch_stats(it, hs ^ 1);
                }
            }
            if (lane == 0) {
                // wait (bounded) for the copies still in flight before the block
                // exits: always, since a consumer may give up after the last copy
                // was issued (after a normal run these phases are complete)
                volatile int no_abort = 0;
                WaitCtl dc{a.err, &no_abort, a.drain_ns};
                if (nkv > 0) wait1(BAR(K_KVFULL), (nkv - 1) & 1, dc);
                for (int s = issued > K_QST ? issued - K_QST : 0; s < issued; ++s)
                    wait1(BAR(K_QFULL + s % K_QST), (s / K_QST) & 1, dc);
            }
        } else {
            // ------------------------------------------------------------ MMA issuers
            // Three issuing warps, so that a wait of one never leaves the tensor
            // pipe without work from the others: warp 2 issues S^T(s) into buffer
            // s%2 once dV(s-2) has read P^T(s-2) out of those columns, warp 3
            // dP^T(s) once dK(s-2) has read dS^T(s-2), and warp 1 dV(s) and dK(s)
            // once the gradient warpgroup has written P^T(s) and dS^T(s).  Each
            // warp runs converged (warp-collective waits), so its operands stay
            // warp-uniform, and one elected lane issues the MMAs and commits.
            const bool leader = elect_one();
            bool ok = true;
            Item x;
            int gs = 0;      // half steps so far (even at the end of a unit)
            if (warp >= 2) {
                constexpr uint32_t idSP = idesc_bf16(128, 64, false);   // N = 64 queries
                // warp 2: S^T = K Q_s^T; warp 3: dP^T = V dO_s^T
                const bool dp = warp == 3;
                const uint64_t dA = sdesc(dp ? sV : sK, 16, 1024);
                const uint64_t dQ0 = sdesc(sQ, 16, 1024) + (dp ? (uint64_t)(HB >> 4) : 0);   // Q_s / dO_s K-major
                const int b_free = dp ? K_DPFREE : K_SFREE, b_done = dp ? K_DP : K_S;
                const uint32_t col = dp ? 64u : 0u;
                Ring<K_QST> rs;
                for (int u = 0; ok && unit_of(u, x); ++u) {
                    if (!waitw(BAR(K_KVFULL), u & 1, wc)) break;
                    for (int s = 0; s < x.ns; ++s, ++gs, rs.next()) {
                        if ((gs >= 2 && !waitw(BAR(b_free + (gs & 1)), ((gs >> 1) - 1) & 1, wc)) ||
                            !waitw(BAR(K_QFULL + rs.st), rs.ph, wc)) {
                            ok = false;
                            break;
                        }
                        const uint32_t tb = tmem + 128u * (uint32_t)(gs & 1) + col;
                        const uint64_t so = (uint64_t)(rs.st * (C::STAGE >> 4));
                        if (leader) {
                            tc_fence_after();
                            ss_seq<0, D, 8192>(tb, dA, dQ0 + so, idSP);
                            mma_commit(BAR(b_done + (gs & 1)));
                        }
                        __syncwarp();
                    }
                    if constexpr (WIN) {
                        if (leader) mma_commit(BAR(K_KVEMPTY));
                        __syncwarp();
                    }
                }
            } else {
                constexpr uint32_t idKV = idesc_bf16(128, D, true);     // dV, dK: B MN-major
                const uint64_t dQmn0 = sdesc(sQ, 8192, 1024);          // Q_s, dO_s MN-major
                const uint32_t tDV = tmem + C::TM_DV, tDK = tmem + C::TM_DK;
                Ring<K_QST> rs;
                int nf = 0;  // units with any step so far (the others have no products)
                for (int u = 0; ok && unit_of(u, x); ++u) {
                    for (int s = 0; s < x.ns; ++s, ++gs, rs.next()) {
                        // P^T(gs) written: warpgroup 0, whose step s = 0 is, has also read the
                        // previous unit's dV, which this unit's first product overwrites
                        if (!waitw(BAR(K_PW + (gs & 1)), (gs >> 1) & 1, wc)) {
                            ok = false;
                            break;
                        }
                        const uint32_t tb = tmem + 128u * (uint32_t)(gs & 1);
                        const uint64_t so = (uint64_t)(rs.st * (C::STAGE >> 4));
                        const uint32_t acc0 = s > 0 ? 1u : 0u;
                        // dV += P^T dO_s as soon as P^T is written, while the gradient
                        // warps compute dS^T; then dK += dS^T Q_s (K = 64 queries: 4 MMAs each)
                        if (leader) {
                            tc_fence_after();
                            ts_mn_seq<0, 4, 0>(tDV, tb, dQmn0 + so + (uint64_t)(HB >> 4), idKV, acc0);
                            mma_commit(BAR(K_SFREE + (gs & 1)));
                            // warpgroup 0 writes dV while warpgroup 1 and the tensor cores are at the last dK
                            if (WIN && s + 1 == x.ns) mma_commit(BAR(K_FINV));
                        }
                        __syncwarp();
                        // ... and before the first dK warpgroup 1 has read the previous unit's
                        if (!waitw(BAR(K_DSW + (gs & 1)), (gs >> 1) & 1, wc) ||
                            (WIN && s == 0 && nf > 0 && !waitw(BAR(K_ACC), (nf - 1) & 1, wc))) {
                            ok = false;
                            break;
                        }
                        if (leader) {
                            tc_fence_after();
                            ts_mn_seq<0, 4, 0>(tDK, tb + 64u, dQmn0 + so, idKV, acc0);
                            // S^T(s) and dP^T(s) completed before the gradient warps read
                            // them, so the stage is free once dV/dK(s) complete
                            mma_commit(BAR(K_QEMPTY + rs.st));
                            mma_commit(BAR(K_DPFREE + (gs & 1)));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (!WIN || x.ns > 0) {
                        if (leader) mma_commit(BAR(K_FIN));
                        __syncwarp();
                        ++nf;
                    }
                }
            }
            if (leader) mma_commit(BAR(K_DRAIN));
            __syncwarp();
            volatile int no_abort = 0;
            WaitCtl dc{a.err, &no_abort, a.drain_ns};
            waitw(BAR(K_DRAIN), 0, dc);
        }
        __syncwarp();
        tc_fence_before();
        asm volatile("barrier.sync 1, %0;" ::"n"(NTHREADS) : "memory");
        if (warp == 0) {
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        }
        return;
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_GRAD));
        // ------------------------------------------------------------ P^T, dS^T
        const int half = (warp - 4) >> 2;           // warpgroup: half steps s with s % 2 == half
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;        // key row of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tb = tmem + lane_off + 128u * (uint32_t)half;
        const float sl2 = a.scale * LOG2E;
        bool ok = true;
        int gi = 0, nf = 0;  // this warpgroup's half steps so far, units with any
        Ring<K_QST> qr;
        if (half) qr.next();
        Item x;
        for (int u = 0; ok && unit_of(u, x); ++u) {
            const KvUnit &w = x.w;
            const int ns = x.ns, piece = x.piece, kpos = w.ks + row;
            Walk it;
            start_walk(it, x);
            for (int i = 0; 2 * i + half < ns; ++i, ++gi, it.next(), qr.next(), qr.next()) {
                const int qa = it.start() + 64 * half, ql = it.len() - 64 * half;
                int sh = 0;
                if constexpr (!WIN) sh = it.shift;
                if (!waitw(BAR(K_S + half), gi & 1, wc) || !waitw(BAR(K_QFULL + qr.st), qr.ph, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t sr[64], pr[64];
                tmem_ld_x64(tb, sr);
                // visible query columns c: c < ql and (not causal or qa + c >= kpos)
                int lo = a.causal ? kpos - sh - qa : 0, hi = ql;
                if constexpr (WIN) {
                    // the query of column c stands at position qa + c + off; a window unit's
                    // keys are seen up to window - 1 behind them, a piece's sinks from there on
                    lo = kpos - a.win.off - qa;
                    if (piece == 0) hi = a.win.window - 1 < ql - 1 - lo ? lo + a.win.window : ql;
                    else lo = kpos < a.win.sinks && a.win.window <= 64 - lo ? lo + a.win.window : 64;
                }
                const float4 *ls4 = reinterpret_cast<const float4 *>(stat + qr.st * 128);   // -lse2
                const float4 *dl4 = ls4 + 16;                                               // -Delta
                // most tiles are visible to the whole warp: no per-element mask there
                const bool full = __all_sync(0xffffffffu, lo <= 0 && hi >= 64);
                // P^T (fp32, kept in place of S^T for dS^T) and its bf16 pairs, stored
                // at once so that their registers are free for dS^T
                {
                    uint32_t pp[32];
#pragma unroll
                    for (int e4 = 0; e4 < 16; ++e4) {
                        const float4 l = ls4[e4];
                        const int c = 4 * e4;
                        float p0, p1, p2, p3;
                        ffma2v(p0, p1, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]), sl2, sl2, l.x, l.y);
                        ffma2v(p2, p3, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]), sl2, sl2, l.z, l.w);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        p2 = ex2(p2);
                        p3 = ex2(p3);
                        if (!full) {
                            p0 = (c >= lo && c < hi) ? p0 : 0.f;
                            p1 = (c + 1 >= lo && c + 1 < hi) ? p1 : 0.f;
                            p2 = (c + 2 >= lo && c + 2 < hi) ? p2 : 0.f;
                            p3 = (c + 3 >= lo && c + 3 < hi) ? p3 : 0.f;
                        }
                        sr[c] = __float_as_uint(p0);
                        sr[c + 1] = __float_as_uint(p1);
                        sr[c + 2] = __float_as_uint(p2);
                        sr[c + 3] = __float_as_uint(p3);
                        pp[2 * e4] = pack_bf16(p0, p1);
                        pp[2 * e4 + 1] = pack_bf16(p2, p3);
                    }
                    tmem_st_x32(tb, pp);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(K_PW + half));   // dV(s) may start
                }
                if (!waitw(BAR(K_DP + half), gi & 1, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_ld_x64(tb + 64u, pr);
                {
                    // dS^T = P^T (dP^T - Delta)
                    uint32_t dd[32];
#pragma unroll
                    for (int e4 = 0; e4 < 16; ++e4) {
                        const float4 d = dl4[e4];
                        const int c = 4 * e4;
                        float t0, t1, t2, t3;
                        fadd2v(t0, t1, __uint_as_float(pr[c]), __uint_as_float(pr[c + 1]), d.x, d.y);
                        fadd2v(t2, t3, __uint_as_float(pr[c + 2]), __uint_as_float(pr[c + 3]), d.z, d.w);
                        fmul2v(t0, t1, t0, t1, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                        fmul2v(t2, t3, t2, t3, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
                        dd[2 * e4] = pack_bf16(t0, t1);
                        dd[2 * e4 + 1] = pack_bf16(t2, t3);
                    }
                    tmem_st_x32(tb + 64u, dd);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(K_DSW + half));
            }
            if (ok && ((WIN && ns == 0) || waitw(BAR(WIN && half == 0 ? K_FINV : K_FIN), nf & 1, wc))) {
                tc_fence_after();
                // half 0 writes dV, half 1 writes dK (times scale)
                bool valid = row < w.kl;
                const float f = half ? a.scale : 1.f;
                const uint32_t tAcc = tmem + lane_off + (half ? C::TM_DK : C::TM_DV);
                const bool a32 = (reinterpret_cast<uintptr_t>(half ? dk : dv) & 31) == 0;
                const int krow = WIN ? dbg_coord(a.err, valid ? kpos : 0, a.Sk)
                                     : dbg_coord(a.err, valid ? slot_pos(g, kpos) : 0, a.S);
                __nv_bfloat16 *orow = (half ? dk : dv) + (((int64_t)w.b * (WIN ? a.Sk : a.S) + krow) * a.Hkv + w.g) * D;
                float *prow = nullptr;   // WIN: a sink's partial gradient
                float odd = 0.f;         // WIN: NaN where an element is not finite
                if constexpr (WIN) {
                    if (valid) prow = partial_row<D>(a, w.b, w.g, piece, kpos, half != 0);
                    valid = valid && !prow && piece == 0;
                }
#pragma unroll (WIN ? 1 : D / 32)
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_x32(tAcc + 32u * c, o);
                    if constexpr (WIN) {
                        if (ns == 0) {           // keys that no row reaches: the accumulators hold nothing
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = 0u;
                        }
                        if (prow) {
                            float4 *dst = reinterpret_cast<float4 *>(prow + 32 * c);
#pragma unroll
                            for (int v4 = 0; v4 < 8; ++v4)
                                dst[v4] = make_float4(__uint_as_float(o[4 * v4]) * f, __uint_as_float(o[4 * v4 + 1]) * f,
                                                      __uint_as_float(o[4 * v4 + 2]) * f, __uint_as_float(o[4 * v4 + 3]) * f);
                        }
                    }
                    if constexpr (WIN) {
                        odd += odd_columns(o);
                        if (a32) {
                            put_row_piece(orow + 32 * c, valid, o, f, lane);
                            continue;
                        }
                    }
                    if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(orow + 32 * c);
#pragma unroll
                        for (int v4 = 0; v4 < 4; ++v4) {
                            uint4 pkt;
                            pkt.x = pack_bf16(__uint_as_float(o[8 * v4 + 0]) * f, __uint_as_float(o[8 * v4 + 1]) * f);
                            pkt.y = pack_bf16(__uint_as_float(o[8 * v4 + 2]) * f, __uint_as_float(o[8 * v4 + 3]) * f);
                            pkt.z = pack_bf16(__uint_as_float(o[8 * v4 + 4]) * f, __uint_as_float(o[8 * v4 + 5]) * f);
                            pkt.w = pack_bf16(__uint_as_float(o[8 * v4 + 6]) * f, __uint_as_float(o[8 * v4 + 7]) * f);
                            dst[v4] = pkt;
                        }
                    }
                }
                if constexpr (WIN) {
                    if (__any_sync(0xffffffffu, (valid || prow) && !(odd == 0.f)) && lane == 0) fixes->note(u, half * 4 + quarter);
                }
            }
            if (WIN && ns > 0) {   // the accumulators may be overwritten
                tc_fence_before();
                __syncwarp();
                if (half && lane == 0) mbar_arrive(BAR(K_ACC));
                ++nf;
            }
        }
        __syncwarp();
        tc_fence_before();
        asm volatile("barrier.sync 1, %0;" ::"n"(NTHREADS) : "memory");
        if constexpr (WIN) {
            if (fixes->count > 0) dkdv_fix<D>(*fixes, a, dk, dv);
        }
        return;
    }
#undef BAR
}

// Delta = rowsum(dO * out) into the workspace
int launch_delta(const BwdPtrs &p, const BwdArgs &a, int D, cudaStream_t st)
{
    const int64_t rows = (int64_t)a.B * a.S * a.Hq;
    int64_t blocks = (rows + 31) / 32;
    const int64_t cap = (int64_t)sm_count() * 8;
    if (blocks > cap) blocks = cap;
    bwd_delta_kernel<<<(unsigned)blocks, 256, 0, st>>>(
        static_cast<const __nv_bfloat16 *>(p.out), static_cast<const __nv_bfloat16 *>(p.dout),
        static_cast<float *>(p.workspace), a.S, a.Hq, D, rows);
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

template <int D>
int launch_window_d(const BwdPtrs &p, BwdArgs a, cudaStream_t st)
{
    CUtensorMap mk, mv, mq, mq64, mdo64;
    PackMaps pm;
    const int pack = a.win.pack, box = pack ? pack : 16;
    if (!make_map(&mk, p.k, a.B, a.Sk, a.Hkv, D, 128) || !make_map(&mv, p.v, a.B, a.Sk, a.Hkv, D, 128) ||
        !make_map(&mq, p.q, a.B, a.S, a.Hq, D, 128) || !make_map(&mq64, p.q, a.B, a.S, a.Hq, D, 64) ||
        !make_map(&mdo64, p.dout, a.B, a.S, a.Hq, D, 64) ||
        !make_map(&pm.k_sinks, p.k, a.B, a.Sk, a.Hkv, D, box) ||
        !make_map(&pm.k_rest, p.k, a.B, a.Sk, a.Hkv, D, 128 - pack) ||
        !make_map(&pm.v_sinks, p.v, a.B, a.Sk, a.Hkv, D, box) ||
        !make_map(&pm.v_rest, p.v, a.B, a.Sk, a.Hkv, D, 128 - pack))
        return CP_ECUDA;
    static std::atomic<bool> attr_done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CP_ECUDA;
    if (dev >= 64 || !attr_done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(bwd_dq_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 DqCfg<D>::SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(bwd_dkdv_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 DkvCfg<D>::SMEM) != cudaSuccess)
            return CP_ECUDA;
        if (dev < 64) attr_done[dev].store(true, std::memory_order_release);
    }
    a.upc = (a.S + T - 1) / T;
    a.tpc = (a.Sk + T - 1) / T;
    a.sp = sink_plan<T, T>(a.win, a.S, a.Sk, a.Hq / a.Hkv, (int64_t)a.B * a.Hkv);
    const int64_t qunits = (int64_t)a.upc * a.B * a.Hq;
    const int64_t kunits = ((int64_t)a.tpc + (int64_t)a.sp.tiles * a.sp.pieces) * a.B * a.Hkv;
    if (qunits > 0x7fffffffLL || kunits > 0x7fffffffLL) return CP_EUNSUPPORTED;
    const int64_t sms = sm_count();
    const int cap = fwd_grid_limit();   // test hook: blocks with many units
    const int64_t most = cap > 0 && cap < sms ? cap : sms;
    float *delta = static_cast<float *>(p.workspace);
    a.delta = delta;
    a.part = delta + bwd_workspace_bytes(a.B, a.Hq, a.S) / 4;
    a.fix = FixArgs{static_cast<const __nv_bfloat16 *>(p.q), static_cast<const __nv_bfloat16 *>(p.k),
                    static_cast<const __nv_bfloat16 *>(p.v), static_cast<const __nv_bfloat16 *>(p.out),
                    static_cast<const __nv_bfloat16 *>(p.dout), p.lse, delta, a.S, a.Sk, a.Hq, a.Hkv, a.scale, a.win};
    __nv_bfloat16 *dk = static_cast<__nv_bfloat16 *>(p.dk), *dv = static_cast<__nv_bfloat16 *>(p.dv);
    a.n_units = (int)qunits;
    a.by_tiles = fast_div((uint32_t)a.upc);
    a.by_heads = fast_div((uint32_t)a.Hq);
    a.by_group = fast_div((uint32_t)(a.Hq / a.Hkv));
    bwd_dq_kernel<D, true><<<(unsigned)(qunits < most ? qunits : most), NTHREADS, DqCfg<D>::SMEM, st>>>(
        mq, mk, mv, mdo64, a, p.lse, delta, static_cast<__nv_bfloat16 *>(p.dq),
        static_cast<const __nv_bfloat16 *>(p.dout), pm);
    if (cudaGetLastError() != cudaSuccess) return CP_ECUDA;
    a.n_units = (int)kunits;
    a.by_tiles = fast_div((uint32_t)a.tpc);
    a.by_heads = fast_div((uint32_t)a.Hkv);
    bwd_dkdv_kernel<D, true><<<(unsigned)(kunits < most ? kunits : most), NTHREADS, DkvCfg<D>::SMEM, st>>>(
        mq64, mk, mv, mdo64, a, p.lse, delta, dk, dv);
    if (cudaGetLastError() != cudaSuccess) return CP_ECUDA;
    return launch_window_sinks<D>(a.part, a.win, a.sp, a.B, a.Hkv, a.Sk, dk, dv, st);
}

template <int D>
int launch_bwd_d(const BwdPtrs &p, BwdArgs a, cudaStream_t st)
{
    CUtensorMap mk, mv, mdo, mq, mq64, mdo64;
    const int R = a.layout == CP_LAYOUT_STRIPED ? a.N : 1;
    if (!make_map(&mk, p.k, a.B, a.S, a.Hkv, D, 128, R) || !make_map(&mv, p.v, a.B, a.S, a.Hkv, D, 128, R) ||
        !make_map(&mdo, p.dout, a.B, a.S, a.Hq, D, 128, R) || !make_map(&mq, p.q, a.B, a.S, a.Hq, D, 128, R) ||
        !make_map(&mq64, p.q, a.B, a.S, a.Hq, D, 64, R) || !make_map(&mdo64, p.dout, a.B, a.S, a.Hq, D, 64, R))
        return CP_ECUDA;
    static bool attr_done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CP_ECUDA;
    if (dev < 64 && !attr_done[dev]) {
        if (cudaFuncSetAttribute(bwd_dq_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 DqCfg<D>::SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(bwd_dkdv_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 DkvCfg<D>::SMEM) != cudaSuccess)
            return CP_ECUDA;
        attr_done[dev] = true;
    }
    const Geom g = make_geom(a.S, a.N, a.layout, a.causal);
    float *delta = static_cast<float *>(p.workspace);
    const int rc = launch_delta(p, a, D, st);
    if (rc) return rc;

    a.upc = (g.clen + T - 1) / T;
    a.tpc = (g.clen + T - 1) / T;
    const int64_t qunits = (int64_t)g.N * g.cpr * a.upc * a.B * a.Hq;
    const int64_t kunits = (int64_t)g.N * g.cpr * a.tpc * a.B * a.Hkv;
    if (qunits > 0x7fffffffLL || kunits > 0x7fffffffLL) return CP_EUNSUPPORTED;
    bwd_dq_kernel<D, false><<<(unsigned)qunits, NTHREADS, DqCfg<D>::SMEM, st>>>(
        mq, mk, mv, mdo, a, p.lse, delta,
        static_cast<__nv_bfloat16 *>(p.dq), static_cast<const __nv_bfloat16 *>(p.dout), NoMaps{});
    if (cudaGetLastError() != cudaSuccess) return CP_ECUDA;
    bwd_dkdv_kernel<D, false><<<(unsigned)kunits, NTHREADS, DkvCfg<D>::SMEM, st>>>(
        mq64, mk, mv, mdo64, a, p.lse, delta, static_cast<__nv_bfloat16 *>(p.dk),
        static_cast<__nv_bfloat16 *>(p.dv));
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace

size_t bwd_workspace_bytes(int B, int Hq, int64_t S)
{
    // Delta: B*Hq*S fp32, rounded up to 256 bytes
    const size_t b = (size_t)B * (size_t)Hq * (size_t)S * 4u;
    return (b + 255u) & ~(size_t)255u;
}

size_t window_bwd_workspace_bytes(int B, int Hq, int Hkv, int Sq, int D, int dtype, const Window &w)
{
    const int64_t heads = (int64_t)B * Hkv;
    const SinkPlan sp = dtype == CP_BF16 ? sink_plan<T, T>(w, Sq, Sq + w.off, Hq / Hkv, heads)
                                         : window_f32_plan(w, Sq, Hq / Hkv, heads);
    size_t b = bwd_workspace_bytes(B, Hq, Sq);
    if (sp.pieces) b += (size_t)B * Hkv * (size_t)window_part_rows(w, sp) * D * sizeof(float);
    return (b + 255u) & ~(size_t)255u;
}

namespace {

BwdArgs bwd_args(const FwdArgs &f)
{
    BwdArgs a;
    a.B = f.B;
    a.Hq = f.Hq;
    a.Hkv = f.Hkv;
    a.S = f.S;
    a.D = f.D;
    a.N = f.N;
    a.causal = f.causal;
    a.layout = f.layout;
    a.scale = f.scale;
    a.upc = a.tpc = 0;
    a.err = f.err;
    a.limit_ns = f.limit_ns;
    a.drain_ns = f.drain_ns;
    a.Sk = 0;
    a.win = Window{0, 0, 0, 0};
    a.sp = SinkPlan{0, 0, 1};
    a.part = a.delta = nullptr;
    a.n_units = 0;
    a.by_tiles = a.by_heads = a.by_group = fast_div(1);
    a.fix = FixArgs{};
    return a;
}

}  // namespace

int launch_window_bwd_bf16(const BwdPtrs &p, const WindowArgs &f, cudaStream_t st)
{
    BwdArgs a = bwd_args(f);
    a.Sk = f.Sk;
    a.win = f.win;
    if (f.D == 64) return launch_window_d<64>(p, a, st);
    if (f.D == 128) return launch_window_d<128>(p, a, st);
    return CP_EUNSUPPORTED;
}

int launch_bwd_bf16(const BwdPtrs &p, const FwdArgs &f, cudaStream_t st)
{
    const BwdArgs a = bwd_args(f);
    if (f.D == 64) return launch_bwd_d<64>(p, a, st);
    if (f.D == 128) return launch_bwd_d<128>(p, a, st);
    return CP_EUNSUPPORTED;
}

}  // namespace cp
