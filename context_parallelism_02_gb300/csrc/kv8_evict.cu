// kv8_evict.cu -- the 8-bit cache cut down to the tokens of the largest accumulated weight.
//
// Per sequence and kv head: kept = the `budget` slots with the largest key, ties to the
// lower slot, in ascending order; key = +infinity for the first and last slots, else the
// slot's mass (NaN counts as the largest).  Two kernels:
//   select  a cluster of blocks per (sequence, kv head), each with a run of its slots in
//           shared memory as 32-bit keys in the order of the floats: mass is read once.
//           Four rounds of 8 bits, each a histogram summed over the cluster through
//           distributed shared memory, find the last key that is kept and how many of its
//           equals; counts by warps of consecutive slots then place the slots.  Bounded by
//           latency: five cluster barriers and the passes over the keys, BATCH loads at a time
//           (rounds of 11 bits save one, but summing 2048 bins costs 4000 cycles each; a run
//           of slots per thread, with its bank conflicts and one load at a time, took 15000
//           cycles for the last two passes and 9 us longer).  8 rows of 65536 slots cut to 16,
//           with next to nothing to move, 17 us; 128 rows of 8192 19.
//   move    a warp per 16 kept tokens and kv head copies their rows of D bytes, K and V, into a
//           block of the other pages, under the largest of their scales.  Bounded by the chain
//           kept slot, page, scale and row, then by HBM (K and V by warps of their own, twice the
//           chains: 1 us longer).  8 rows of 65536 slots to 16384: 14 us on top of the selection.
#include <cooperative_groups.h>

#include <atomic>

#include "kernels.h"
#include "kv8.cuh"

namespace cp {

namespace {

namespace cg = cooperative_groups;

constexpr int THREADS = 512, NWARP = THREADS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_KEYS = 49152;    // keys of a block that lie in shared memory (192 KB)
constexpr int MOVE_WARPS = 8;

// Order of floats as unsigned integers, -0 as 0, NaN above all but the slots kept anyway.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (x != x) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int BINS = 256, ROUNDS = 4;
constexpr int BATCH = 16;          // slots of a thread whose loads are in flight together
struct Shared {
    uint32_t hist[ROUNDS][BINS];   // a round each: the cluster may still read one while the next fills
    uint32_t before[2];            // in the blocks of lower rank: keys above the last kept one, equals
    uint32_t warp[NWARP][2];
    uint32_t prefix, want;         // digits found so far; equals of them still to take
};

// Sum over the block's threads of lower index, of two counts at once.
__device__ __forceinline__ void scan2(Shared &sm, uint32_t (&v)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t in[2] = {v[0], v[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, in[i], o);
            if (lane >= o) in[i] += x;
        }
    if (lane == 31) sm.warp[warp][0] = in[0], sm.warp[warp][1] = in[1];
    __syncthreads();
    uint32_t base[2] = {0, 0};
    for (int w = 0; w < warp; ++w) base[0] += sm.warp[w][0], base[1] += sm.warp[w][1];
    v[0] = base[0] + in[0] - v[0];
    v[1] = base[1] + in[1] - v[1];
}

__global__ void __launch_bounds__(THREADS) kv8_select_kernel(Kv8EvictArgs a, int in_shared)
{
    extern __shared__ uint32_t keys[];
    __shared__ Shared sm;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const unsigned row = blockIdx.x / (unsigned)C;           // (sequence, kv head)
    const int b = (int)(row / (unsigned)a.pool.Hkv);
    kv4_begin();
    const int len = kv4_len(a.pool, b);
    const int64_t cap = (int64_t)a.pool.max_pages << a.pool.page_shift;
    const int64_t cap_to = (int64_t)a.max_to << a.pool.page_shift;
    const float *mass = a.mass + (int64_t)row * cap;
    int32_t *kept = a.kept + (int64_t)row * a.budget;
    float *mass_to = a.mass_to ? a.mass_to + (int64_t)row * cap_to : nullptr;
    const int n = len < a.budget ? len : a.budget;           // slots that are kept
    // what lies behind them
    for (int64_t i = n + (int64_t)rank * THREADS + threadIdx.x; i < (a.budget > cap_to ? a.budget : cap_to); i += (int64_t)C * THREADS) {
        if (i < a.budget) kept[i] = -1;
        if (mass_to && i < cap_to) mass_to[i] = 0.f;
    }
    if (rank == 0 && threadIdx.x == 0 && row % (unsigned)a.pool.Hkv == 0) a.lens_to[b] = n;
    // this block's run of slots, and in it the warp's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int run = (len + C - 1) / C, s0 = min(rank * run, len), s1 = min(s0 + run, len);
    const int seg = ((s1 - s0 + NWARP - 1) / NWARP + 31) & ~31;
    const int w0 = min(s0 + warp * seg, s1), w1 = min(w0 + seg, s1);
    if (len <= a.budget) {                                   // all of them (the same in the whole cluster)
        for (int s = s0 + threadIdx.x; s < s1; s += THREADS) {
            kept[s] = s;
            if (mass_to) mass_to[s] = mass[s];
        }
        return;
    }
    auto key_from = [&](int s, float x) -> uint32_t {
        return s < a.first || s >= len - a.last ? 0xffffffffu : key_of(x);
    };
    // f(slot, key, whether it is there) for the warp's slots, 32 consecutive ones at a time
    auto each_key = [&](auto f) {
        for (int t = w0; t < w1; t += 32 * BATCH) {
            uint32_t k[BATCH];
            if (in_shared) {
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int s = t + 32 * i + lane;
                    k[i] = s < w1 ? keys[s - s0] : 0u;
                }
            } else {
                float x[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) x[i] = t + 32 * i + lane < w1 ? mass[t + 32 * i + lane] : 0.f;
#pragma unroll
                for (int i = 0; i < BATCH; ++i) k[i] = key_from(t + 32 * i + lane, x[i]);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (t + 32 * i < w1) f(t + 32 * i + lane, k[i], t + 32 * i + lane < w1);
        }
    };
    if (in_shared) {
        for (int t = w0; t < w1; t += 32 * BATCH) {
            float x[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) x[i] = t + 32 * i + lane < w1 ? mass[t + 32 * i + lane] : 0.f;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int s = t + 32 * i + lane;
                if (s < w1) keys[s - s0] = key_from(s, x[i]);
            }
        }
    }
    if (threadIdx.x == 0) sm.prefix = 0, sm.want = (uint32_t)n, sm.before[0] = 0;
    for (int i = threadIdx.x; i < ROUNDS * BINS; i += THREADS) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    for (int round = 0; round < ROUNDS; ++round) {
        const int shift = 24 - 8 * round;
        uint32_t *hist = sm.hist[round];
        const uint32_t prefix = sm.prefix, want = sm.want;
        each_key([&](int, uint32_t k, bool there) {
            if (there && (round == 0 || k >> (shift + 8) == prefix)) atomicAdd(&hist[k >> shift & 255u], 1u);
        });
        cl.sync();
        // the digit that the want-th largest key has: thread i sums bin 255 - i over the cluster
        const int bin = BINS - 1 - (int)threadIdx.x;
        uint32_t v[2] = {0, 0};
        if (bin >= 0) {
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) {          // all loads in flight
                const uint32_t x = r < C ? cl.map_shared_rank(hist, r)[bin] : 0u;
                v[0] += x;
                v[1] += r < rank ? x : 0u;
            }
        }
        const uint32_t here = v[0], lower = v[1];
        scan2(sm, v);                                        // keys in higher bins
        if (v[0] < want && v[0] + here >= want) {            // one thread
            sm.prefix = prefix << 8 | (uint32_t)bin;
            sm.want = want - v[0];
            sm.before[0] += v[1];
            sm.before[1] = lower;
        }
        __syncthreads();
    }
    cl.barrier_arrive();                                     // this block has read the others' histograms
    // The last kept key is `last`; `equals` of those like it are kept, from the lowest slot on.
    const uint32_t last = sm.prefix, equals = sm.want;
    uint32_t at[2] = {0, 0};                                 // keys above it, equals: in the warp's slots
    each_key([&](int, uint32_t k, bool there) {
        at[0] += __popc(__ballot_sync(0xffffffffu, there && k > last));
        at[1] += __popc(__ballot_sync(0xffffffffu, there && k == last));
    });
    if (lane == 0) sm.warp[warp][0] = at[0], sm.warp[warp][1] = at[1];
    __syncthreads();
    // ... and before them
    at[0] = sm.before[0], at[1] = sm.before[1];
    for (int w = 0; w < warp; ++w) at[0] += sm.warp[w][0], at[1] += sm.warp[w][1];
    const unsigned lower = (1u << lane) - 1u;
    for (int t = w0; t < w1; t += 32 * BATCH) {
        float x[BATCH];                                      // mass again, for mass_to (in L2)
#pragma unroll
        for (int i = 0; i < BATCH; ++i) x[i] = t + 32 * i + lane < w1 ? mass[t + 32 * i + lane] : 0.f;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int s = t + 32 * i + lane;
            if (t + 32 * i >= w1) break;
            const bool there = s < w1;
            const uint32_t k = in_shared ? (there ? keys[s - s0] : 0u) : key_from(s, x[i]);
            const unsigned gt = __ballot_sync(0xffffffffu, there && k > last), eq = __ballot_sync(0xffffffffu, there && k == last);
            const uint32_t ties = at[1] + __popc(eq & lower);
            if (there && (k > last || (k == last && ties < equals))) {
                const uint32_t to = at[0] + __popc(gt & lower) + min(ties, equals);
                kept[to] = s;
                if (mass_to) mass_to[to] = x[i];
            }
            at[0] += __popc(gt);
            at[1] += __popc(eq);
        }
    }
    cl.barrier_wait();                                       // the others have read this one's
}

// 16 kept tokens of one kv head, K and V.
template <int D>
__global__ void __launch_bounds__(MOVE_WARPS * 32) kv8_move_kernel(Kv8EvictArgs a, FastDiv by_heads, FastDiv by_blocks, int units)
{
    constexpr int LANES = D / 16, ROWS = 32 / LANES, N = 16 / ROWS;
    const int lane = threadIdx.x & 31;
    kv4_begin();
    const int64_t unit = (int64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    if (unit >= units) return;
    const unsigned x0 = (unsigned)unit, y0 = by_heads.div(x0);
    const int h = (int)(x0 - y0 * by_heads.d), b = (int)by_blocks.div(y0), t = (int)(y0 - (unsigned)b * by_blocks.d);
    const int64_t i0 = (int64_t)t * KV8_BLOCK;
    // where it goes
    const int64_t lp = i0 >> a.pool.page_shift;
    const int id_to = lp < a.max_to ? a.to[(int64_t)b * a.max_to + lp] : -1;
    // lane r < 16: where token r of the block comes from
    int slot = -1;
    if (lane < KV8_BLOCK && i0 + lane < a.budget) slot = a.kept[((int64_t)b * a.pool.Hkv + h) * a.budget + i0 + lane];
    const int64_t v_bytes = (int64_t)D << a.pool.page_shift, v_scales = (int64_t)1 << (a.pool.page_shift - 4);
    const uint8_t *src = nullptr;          // K's row; V's lies v_bytes behind it
    float scale[2] = {0.f, 0.f};
    if (slot >= 0) {
        const int id = kv4_page(a.pool, b, slot >> a.pool.page_shift);
        if (id >= 0) {
            const int at = slot & ((1 << a.pool.page_shift) - 1);
            src = kv8_row<D>(a.pool, id, h, 0, at);
            const float *s = kv8_scale(a.pool, id, h, 0, at);
            scale[0] = s[0];
            scale[1] = s[v_scales];
        }
    }
    const unsigned there = __ballot_sync(0xffffffffu, slot >= 0);
    if (!there) return;
    uint4 x[2][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = lane / LANES + i * ROWS;
        const uint8_t *p = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), r));
#pragma unroll
        for (int w = 0; w < 2; ++w)
            x[w][i] = p ? *reinterpret_cast<const uint4 *>(p + w * v_bytes + lane % LANES * 16) : make_uint4(0, 0, 0, 0);
    }
    if (id_to < 0 || id_to >= a.pool.n_pages) {
        if (lane == 0) kv4_report(a.pool.err);
        return;
    }
    const int at = (int)(i0 & ((1 << a.pool.page_shift) - 1));
    uint8_t *dst = kv8_row<D>(a.pool, id_to, h, 0, at);
    float *scale_to = kv8_scale(a.pool, id_to, h, 0, at);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float top = scale[w];
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!(top > 0.f)) top = kv8_scale_of(0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = lane / LANES + i * ROWS;
            const float f = __shfl_sync(0xffffffffu, scale[w], r) / top;             // 0 for a token whose page is not there
            if (!(there >> r & 1u)) continue;
            uint4 &y = x[w][i];
            if (f != 1.f) {
                y.x = kv8_shrink(y.x, f);
                y.y = kv8_shrink(y.y, f);
                y.z = kv8_shrink(y.z, f);
                y.w = kv8_shrink(y.w, f);
            }
            *reinterpret_cast<uint4 *>(dst + w * v_bytes + r * D + lane % LANES * 16) = y;
        }
        if (lane == 0) scale_to[w * v_scales] = top;
    }
}

}  // namespace

int launch_kv8_evict(const Kv8EvictArgs &a, int D, cudaStream_t st)
{
    const int64_t rows = (int64_t)a.B * a.pool.Hkv, cap = (int64_t)a.pool.max_pages << a.pool.page_shift;
    const int64_t blocks = ((int64_t)a.budget + KV8_BLOCK - 1) / KV8_BLOCK;
    const __int128 units = (__int128)rows * blocks;
    if (cap > 0x7fffffffLL || rows * MAX_CLUSTER > 0x7fffffffLL || units > 0x7fffffff)
        return CP_EUNSUPPORTED;
    // blocks of a cluster: as many as leave each about 2048 slots, but no more than run at
    // once, two to an SM (128 rows of 8192 slots: 19 us with 4 blocks each, 18 with 2)
    int C = 1;
    while (C < MAX_CLUSTER && cap > (int64_t)C * 2048 && rows * C <= sm_count()) C *= 2;
    const int64_t run = (cap + C - 1) / C;
    const int in_shared = run <= MAX_KEYS;
    const size_t smem = in_shared ? (size_t)run * 4 : 0;
    static std::atomic<bool> attr_done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CP_ECUDA;
    if (dev >= 64 || !attr_done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kv8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_KEYS * 4) != cudaSuccess)
            return CP_ECUDA;
        if (dev < 64) attr_done[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kv8_select_kernel, a, in_shared) != cudaSuccess) return CP_ECUDA;
    const unsigned grid = (unsigned)(((int64_t)units + MOVE_WARPS - 1) / MOVE_WARPS);
    const cudaError_t rc = kv4_launch(D == 64 ? kv8_move_kernel<64> : kv8_move_kernel<128>, grid, MOVE_WARPS * 32, 0, st, a,
                                      fast_div((uint32_t)a.pool.Hkv), fast_div((uint32_t)blocks), (int)units);
    return rc == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace cp
