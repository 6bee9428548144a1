// kv8_evict.cu -- the 8-bit cache cut down to the tokens of the largest accumulated weight.
//
// Per sequence and kv head: kept = the `budget` slots with the largest key, ties to the
// lower slot, in ascending order; key = +infinity for the first and last slots, else the
// slot's mass (NaN counts as the largest).  Two kernels:
//   select  a cluster of blocks per (sequence, kv head), each with a run of its slots in
//           shared memory as 32-bit keys in the order of the floats: mass is read once.
//           Three rounds of 11, 11 and 10 bits, each a histogram summed over the cluster
//           through distributed shared memory, find the last key that is kept and how many
//           of its equals; prefix sums over runs then place the slots.  Bounded by latency
//           (five cluster barriers; with rounds of 8 bits, where a float's exponents fall on
//           few bins, and ten barriers 8 rows of 65536 slots took 26 us).
//   move    a warp per 16 kept tokens, kv head and K or V copies their rows of D bytes into
//           a block of the other pages, under the largest of their scales.  Bounded by HBM.
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

constexpr int BINS = 2048;
struct Shared {
    uint32_t hist[3][BINS];        // a round each: the cluster may still read one while the next fills
    uint32_t counts[2];            // of the block: keys above the last kept one, equals
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
    // this block's run of slots
    const int run = (len + C - 1) / C, s0 = min(rank * run, len), s1 = min(s0 + run, len);
    if (len <= a.budget) {                                   // all of them (the same in the whole cluster)
        for (int s = s0 + threadIdx.x; s < s1; s += THREADS) {
            kept[s] = s;
            if (mass_to) mass_to[s] = mass[s];
        }
        return;
    }
    auto key_at = [&](int s) -> uint32_t {
        if (s < a.first || s >= len - a.last) return 0xffffffffu;
        return key_of(mass[s]);
    };
    auto key = [&](int s) -> uint32_t { return in_shared ? keys[s - s0] : key_at(s); };
    if (in_shared) {
        constexpr int BATCH = 8;                             // loads in flight of a thread
        for (int t = s0 + threadIdx.x; t < s1; t += BATCH * THREADS) {
            float x[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) x[i] = t + i * THREADS < s1 ? mass[t + i * THREADS] : 0.f;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int s = t + i * THREADS;
                if (s < s1) keys[s - s0] = s < a.first || s >= len - a.last ? 0xffffffffu : key_of(x[i]);
            }
        }
    }
    if (threadIdx.x == 0) sm.prefix = 0, sm.want = (uint32_t)n;
    for (int i = threadIdx.x; i < 3 * BINS; i += THREADS) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    // 11, 11 and 10 bits from the top
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
        uint32_t *hist = sm.hist[round];
        const uint32_t prefix = sm.prefix, want = sm.want;
#pragma unroll 4
        for (int s = s0 + threadIdx.x; s < s1; s += THREADS) {
            const uint32_t k = key(s);
            if (round == 0 || k >> (shift + bits) == prefix) atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1u);
        }
        cl.sync();
        // the digit that the want-th largest key has: a thread sums PER neighbouring bins over
        // the cluster, from the top, and the one where the count passes `want` looks further
        constexpr int PER = BINS / THREADS;
        const int top = (1 << bits) - 1 - (int)threadIdx.x * PER;   // its highest bin (negative: none)
        uint32_t v[PER] = {}, above[2] = {0, 0};
        if (top >= 0) {
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) {                 // all loads in flight
                if (r >= C) continue;
                const uint4 x = *reinterpret_cast<const uint4 *>(cl.map_shared_rank(hist, r) + top - (PER - 1));
                v[0] += x.w, v[1] += x.z, v[2] += x.y, v[3] += x.x;
            }
        }
        static_assert(PER == 4, "one uint4 a thread");
#pragma unroll
        for (int e = 0; e < PER; ++e) above[0] += v[e];
        const uint32_t sum = above[0];
        scan2(sm, above);                                           // keys in higher bins
        if (above[0] < want && above[0] + sum >= want) {            // one thread
            uint32_t at = above[0];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                if (at < want && at + v[e] >= want) {
                    sm.prefix = prefix << bits | (uint32_t)(top - e);
                    sm.want = want - at;
                }
                at += v[e];
            }
        }
        __syncthreads();
    }
    // The last kept key is `last`; `equals` of those like it are kept, from the lowest slot on.
    const uint32_t last = sm.prefix, equals = sm.want;
    // a thread takes a run of neighbouring slots
    const int per = (s1 - s0 + THREADS - 1) / THREADS;
    const int t0 = min(s0 + (int)threadIdx.x * per, s1), t1 = min(t0 + per, s1);
    uint32_t count[2] = {0, 0};
    for (int s = t0; s < t1; ++s) {
        const uint32_t k = key(s);
        count[0] += k > last;
        count[1] += k == last;
    }
    uint32_t at[2] = {count[0], count[1]};
    scan2(sm, at);
    if (threadIdx.x == THREADS - 1) sm.counts[0] = at[0] + count[0], sm.counts[1] = at[1] + count[1];
    cl.sync();
    for (int r = 0; r < rank; ++r) {
        const uint32_t *other = cl.map_shared_rank(sm.counts, r);
        at[0] += other[0];
        at[1] += other[1];
    }
    for (int s = t0; s < t1; ++s) {
        const uint32_t k = key(s);
        if (k > last || (k == last && at[1] < equals)) {
            const uint32_t i = at[0] + min(at[1], equals);
            kept[i] = s;
            if (mass_to) mass_to[i] = mass[s];
        }
        at[0] += k > last;
        at[1] += k == last;
    }
    cl.sync();                                               // counts are read by other blocks
}

// 16 kept tokens of one kv head, K or V.
template <int D>
__global__ void __launch_bounds__(MOVE_WARPS * 32) kv8_move_kernel(Kv8EvictArgs a, int blocks, int64_t units)
{
    constexpr int LANES = D / 16, ROWS = 32 / LANES, N = 16 / ROWS;
    const int lane = threadIdx.x & 31;
    kv4_begin();
    const int64_t unit = (int64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    if (unit >= units) return;
    const int which = (int)(unit & 1);
    int64_t rest = unit >> 1;
    const int h = (int)(rest % a.pool.Hkv);
    rest /= a.pool.Hkv;
    const int t = (int)(rest % blocks), b = (int)(rest / blocks);
    const int64_t i0 = (int64_t)t * KV8_BLOCK;
    // lane r < 16: where token r of the block comes from
    int slot = -1;
    if (lane < KV8_BLOCK && i0 + lane < a.budget) slot = a.kept[((int64_t)b * a.pool.Hkv + h) * a.budget + i0 + lane];
    const uint8_t *src = nullptr;
    float scale = 0.f;
    if (slot >= 0) {
        const int id = kv4_page(a.pool, b, slot >> a.pool.page_shift);
        if (id >= 0) {
            const int at = slot & ((1 << a.pool.page_shift) - 1);
            src = kv8_row<D>(a.pool, id, h, which, at);
            scale = *kv8_scale(a.pool, id, h, which, at);
        }
    }
    const unsigned there = __ballot_sync(0xffffffffu, slot >= 0);
    if (!there) return;
    float top = scale;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // where it goes
    int64_t lp = i0 >> a.pool.page_shift;
    int id = lp < a.max_to ? a.to[(int64_t)b * a.max_to + lp] : -1;
    if (id < 0 || id >= a.pool.n_pages) {
        if (lane == 0) kv4_report(a.pool.err);
        return;
    }
    const int at = (int)(i0 & ((1 << a.pool.page_shift) - 1));
    uint8_t *dst = kv8_row<D>(a.pool, id, h, which, at);
    uint4 x[N];
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = lane / LANES + i * ROWS;
        const uint8_t *p = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), r));
        f[i] = __shfl_sync(0xffffffffu, scale, r) / top;
        x[i] = p ? *reinterpret_cast<const uint4 *>(p + lane % LANES * 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = lane / LANES + i * ROWS;
        if (!(there >> r & 1u)) continue;
        if (f[i] != 1.f) {
            x[i].x = kv8_shrink(x[i].x, f[i]);
            x[i].y = kv8_shrink(x[i].y, f[i]);
            x[i].z = kv8_shrink(x[i].z, f[i]);
            x[i].w = kv8_shrink(x[i].w, f[i]);
        }
        *reinterpret_cast<uint4 *>(dst + r * D + lane % LANES * 16) = x[i];
    }
    if (lane == 0) *kv8_scale(a.pool, id, h, which, at) = top;
}

}  // namespace

int launch_kv8_evict(const Kv8EvictArgs &a, int D, cudaStream_t st)
{
    const int64_t rows = (int64_t)a.B * a.pool.Hkv, cap = (int64_t)a.pool.max_pages << a.pool.page_shift;
    const int64_t blocks = ((int64_t)a.budget + KV8_BLOCK - 1) / KV8_BLOCK;
    const __int128 units = (__int128)rows * blocks * 2;
    if (cap > 0x7fffffffLL || rows * MAX_CLUSTER > 0x7fffffffLL || units > (__int128)0x7fffffff * MOVE_WARPS)
        return CP_EUNSUPPORTED;
    // blocks of a cluster: as many as leave each about 2048 slots
    int C = 1;
    while (C < MAX_CLUSTER && cap > (int64_t)C * 2048) C *= 2;
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
                                      (int)blocks, (int64_t)units);
    return rc == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace cp
