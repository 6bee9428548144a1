// kv_line.cuh -- what the attention kernels of the paged caches share: the schedule
// that cuts a batch of sequences of any lengths into equal stretches of token blocks,
// the join of the pieces, and the instructions of mma.m16n8k16.
//
// All items' blocks of 16 tokens form one line, batch by batch and item by item, and
// every warp of a grid that just fills the GPU takes an equal stretch of it.  A cache's
// argument type A has rows, pool, ws, out, out_f32 and lse, and says with Line<A> how
// many blocks an item of sequence b has and what it costs beyond them.
#pragma once

#include "kv4.cuh"
#include "tc_helpers.cuh"

namespace cp {

// Of the arguments A: PAD, LEAST, NEXT_EARLY and blocks<EARLY>(a, b), at least 1 (EARLY: by a
// kernel that has not waited yet, see kv4_len).
//   PAD    what an item costs beyond its blocks, in blocks
//   LEAST  blocks that a warp takes at least
//   NEXT_EARLY  the join lets the next kernel start before its own wait.  That is worth 1 us
//          of 33 to the 4-bit cache (64 ragged sequences up to 8192 tokens: 32.1 us, behind
//          the wait 33.1; its other cases do not tell).  The 8-bit cache's attention fills
//          the registers of the SMs: a next call's blocks take what the join's are waiting
//          for (8 x 16384 tokens, D = 64, 2 query heads a kv head: 28 us behind the wait, 42
//          before it).
template <typename A>
struct Line;

namespace {

constexpr float LN2 = 0.69314718055994530942f, LOG2E = 1.44269504088896340736f;

// D += A B, fp16 operands, fp32 accumulators, 16 x 8 x 16.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 x 8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t h2(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }

__device__ __forceinline__ float ex2(float x) { return tc::ex2(x); }

// What a row index of an item stands for.  Items are numbered batch by batch;
// within one, token (sparse launches only), row tile and kv head.
struct Item {
    int b, j0, tile, h;   // j0: the token (sparse), else 0
};

struct Shape {
    int group;       // query heads per kv head
    int rows;        // rows of an item's kv head: tokens x group, or group (sparse)
    int tiles;       // row tiles
    int per_batch;   // items of a sequence
};

__device__ __forceinline__ Item decode_item(const Shape &s, int Hkv, int b, int i)
{
    Item it;
    it.b = b;
    const unsigned r = (unsigned)i / (unsigned)Hkv;   // (token, row tile)
    it.h = i - (int)r * Hkv;
    it.j0 = s.tiles == 1 ? (int)r : (int)(r / (unsigned)s.tiles);
    it.tile = (int)r - it.j0 * s.tiles;
    return it;
}

// First slot of a block that is not there: past every row's limit.
constexpr int NO_SLOT = 0x7ffffff0;

template <int D, int NT>
struct Part {              // a piece's result in the workspace
    static constexpr int FLOATS = NT * 8 * (D + 2);   // m, l of each row, then the rows
};

// Rows of warps' parts that the workspace has room for (twice); kv8_attn.cu has room for more of
// 64 elements.
constexpr int MAX_ROWS = 2560 * 8;
// Stretches, one a warp, are fewer than this: Cuts multiplies two numbers below theirs in 32 bits.
constexpr int MAX_STRETCHES = 1 << 16;
static_assert(MAX_ROWS / 8 < MAX_STRETCHES, "a warp's part has 8 rows at least");

// A walk over the pieces of a warp's stretch.
struct Walk {
    int b, i;        // sequence, item of it
    int nb;          // the item's blocks
    int t0, t1;      // the piece: blocks [t0, t1) of the item, none if t0 >= t1
    int64_t left;    // what remains of the stretch, from t0 on
    __device__ __forceinline__ bool valid() const { return left > 0; }
    __device__ __forceinline__ void cut() { t1 = left < nb - t0 ? t0 + (int)left : nb; }
    template <typename A>
    __device__ __forceinline__ void next(const A &a, int per_batch)
    {
        left -= nb + Line<A>::PAD - t0;
        if (left <= 0) return;
        t0 = 0;
        if (++i == per_batch) {
            i = 0;
            ++b;
            nb = Line<A>::template blocks<false>(a, b);
        }
        cut();
    }
};

// Over the batch, by a warp of the join, before its wait: the extent of one item of
// every sequence, and of those before sequence `upto`.
template <typename A>
__device__ __forceinline__ void count_blocks(const A &a, int upto, int64_t &all, int64_t &before)
{
    all = before = 0;
    for (int b = threadIdx.x & 31; b < a.rows.B; b += 32) {
        const int n = Line<A>::template blocks<true>(a, b) + Line<A>::PAD;
        all += n;
        if (b < upto) before += n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
}

// a / b, by the 32-bit division (a fifth of the 64-bit one's chain of instructions)
// where both fit, as they do but for lines of 2^31 blocks.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    return (a | b) >> 31 == 0 ? (int64_t)((unsigned)a / (unsigned)b) : a / b;
}

// The line of `all` blocks in equal stretches: how many there are (a warp takes at
// least `least` blocks), where stretch c begins (floor(all c / n)), and which one holds
// position f.
struct Cuts {
    int64_t each;     // all / n
    int n, over;      // all % n
    float rate;       // n / all
    __device__ __forceinline__ Cuts(int64_t all, int warps, int least)
    {
        const int64_t most = all / least;
        n = most < 1 ? 1 : most < warps ? (int)most : warps;
        each = divide(all, n);
        over = (int)(all - each * n);
        rate = (float)n / (float)all;
    }
    __device__ __forceinline__ int64_t begin(int c) const
    {
        return each * c + (unsigned)over * (unsigned)c / (unsigned)n;   // over and c below MAX_STRETCHES
    }
    __device__ __forceinline__ int at(int64_t f) const
    {
        int c = min((int)((float)f * rate), n - 1);   // off by one at most
        while (c > 0 && begin(c) > f) --c;
        while (c + 1 < n && begin(c + 1) <= f) ++c;
        return c;
    }
};

// Where stretch `self` begins: the extents of all items, then the sequence.  False: there is
// no such stretch.  Every warp of the block calls it; it passes a __syncthreads.
template <typename A>
__device__ __forceinline__ bool start_of_stretch(const A &a, const Shape &sh, int warps, int self, Walk &at)
{
    constexpr int PAD = Line<A>::PAD;
    const int B = a.rows.B, lane = threadIdx.x & 31;
    int64_t all = 0;
    int one = 0;                              // the lane's sequence of the stretch of 32 in hand
    for (int b = lane; b < B; b += 32) {
        one = Line<A>::template blocks<false>(a, b) + PAD;
        all += one;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    all *= sh.per_batch;
    const Cuts cuts(all, warps, Line<A>::LEAST);
    __syncthreads();
    if (self >= cuts.n) return false;
    const int64_t f0 = cuts.begin(self);
    int64_t rest = 0;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        if (B > 32) one = b < B ? Line<A>::template blocks<false>(a, b) + PAD : 0;
        else if (b >= B) one = 0;
        int64_t upto = one;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const int64_t here = __shfl_sync(0xffffffffu, upto, 31) * sh.per_batch;
        if (f0 - rest >= here) {
            rest += here;
            continue;
        }
        const unsigned past = __ballot_sync(0xffffffffu, f0 - rest >= upto * sh.per_batch);
        const int x = __popc(past);           // sequences of these 32 that end before f0
        at.b = b0 + x;
        at.nb = __shfl_sync(0xffffffffu, one, x) - PAD;
        rest = f0 - rest - __shfl_sync(0xffffffffu, upto - one, x) * sh.per_batch;
        break;
    }
    at.i = (int)divide(rest, at.nb + PAD);
    at.t0 = (int)(rest - (int64_t)at.i * (at.nb + PAD));
    at.left = cuts.begin(self + 1) - f0;
    at.cut();
    return true;
}

// One output row's four elements.
template <typename A>
__device__ __forceinline__ void put_out(const A &a, int64_t at, float4 o)
{
    if (a.out_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = o;
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
            make_uint2(tc::pack_bf16(o.x, o.y), tc::pack_bf16(o.z, o.w));
}

// Line `at` of an array of `bytes` bytes into L2.
__device__ __forceinline__ void prefetch(const void *p, int64_t at, int64_t bytes)
{
    if (at < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p) + at));
}

__device__ __forceinline__ uint64_t policy_evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// The warps' states of a block that has an item to itself.
template <int D, int NT, int W>
struct Joined {
    float o[W][NT * 8][D];
    float m[W][NT * 8], l[W][NT * 8];
};

// Joins the pieces of the items that were cut: one block per output row.  The
// parts are read JOIN_DEEP at a time by each of JW warps, so that a row of many pieces (one
// long sequence: up to all warps of the grid) costs a few memory latencies.
template <typename A, int D, int NT, int JW, int JOIN_DEEP>
__global__ void __launch_bounds__(JW * 32) kv_join_kernel(A a, Shape sh, int warps)
{
    constexpr int E = D / 32;
    __shared__ float sm_m[JW], sm_l[JW];
    __shared__ __align__(16) float sm_o[JW][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned item = blockIdx.x / (unsigned)sh.rows, heads = sh.per_batch / sh.tiles;
    const int rr_all = (int)(blockIdx.x - item * sh.rows);
    const int b = (int)(item / heads), x = (int)(item - b * heads);   // x: (token, kv head)
    // The lengths, and nothing else, are read before the wait: the attention kernel triggers
    // after its own, so this grid starts when what wrote them is complete.  The loads are
    // coherent at the GPU's scope: this SM may hold an older line of them.  (Behind the
    // wait they cost a call 2 us: 131072 tokens 39.6 instead of 37.8.)
    if (Line<A>::NEXT_EARLY) kv4_trigger();
    int64_t all, before;
    count_blocks(a, b, all, before);
    all *= sh.per_batch;
    const Cuts cuts(all, warps, Line<A>::LEAST);
    const int nb = Line<A>::template blocks<true>(a, b);
    // the item of this row: token, row tile, kv head
    const int tile = rr_all / (NT * 8), row = rr_all % (NT * 8);
    const int h = x % a.pool.Hkv, j0 = x / a.pool.Hkv;
    const int i = (j0 * sh.tiles + tile) * a.pool.Hkv + h;
    const int64_t f = before * sh.per_batch + (int64_t)i * (nb + Line<A>::PAD);
    const int c0 = cuts.at(f), c1 = cuts.at(f + nb - 1);
    kv4_wait();
    if (!Line<A>::NEXT_EARLY) kv4_trigger();
    if (c0 == c1) return;
    const float *ws = static_cast<const float *>(a.ws);
    float m = -INFINITY, l = 0.f;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int c = c0 + warp * JOIN_DEEP; c <= c1; c += JW * JOIN_DEEP) {
        float pm[JOIN_DEEP], pl[JOIN_DEEP], v[JOIN_DEEP][E], mn = m;
#pragma unroll
        for (int u = 0; u < JOIN_DEEP; ++u) {
            pm[u] = -INFINITY;
            pl[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
            if (c + u > c1) continue;
            const float *part = ws + (2 * (int64_t)(c + u) + (c + u == c0 ? 1 : 0)) * Part<D, NT>::FLOATS;
            pm[u] = part[row];
            pl[u] = part[8 * NT + row];
            if (E == 4) {
                const float4 w = *reinterpret_cast<const float4 *>(part + 16 * NT + row * D + lane * 4);
                v[u][0] = w.x, v[u][1] = w.y, v[u][E - 2] = w.z, v[u][E - 1] = w.w;
            } else {
                const float2 w = *reinterpret_cast<const float2 *>(part + 16 * NT + row * D + lane * 2);
                v[u][0] = w.x, v[u][1] = w.y;
            }
        }
#pragma unroll
        for (int u = 0; u < JOIN_DEEP; ++u) mn = fmaxf(mn, pm[u]);
        const float fa = m == mn ? 1.f : ex2(m - mn);
        l *= fa;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= fa;
#pragma unroll
        for (int u = 0; u < JOIN_DEEP; ++u) {
            const float fu = pm[u] == mn ? 1.f : ex2(pm[u] - mn);
            l = fmaf(pl[u], fu, l);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(v[u][e], fu, o[e]);
        }
        m = mn;
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D) return;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < JW; ++w) m = fmaxf(m, sm_m[w]);
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < JW; ++w) {
        const float fw = sm_m[w] == m ? 1.f : ex2(sm_m[w] - m);
        l = fmaf(fw, sm_l[w], l);
        r = fmaf(fw, sm_o[w][threadIdx.x], r);
    }
    const int j = j0 + rr_all / sh.group, head = h * sh.group + rr_all % sh.group;
    const bool empty = l == 0.f;
    r *= empty ? 0.f : 1.f / l;
    const int64_t at = (((int64_t)b * a.rows.n + j) * a.rows.Hq + head) * D + threadIdx.x;
    if (a.out_f32) static_cast<float *>(a.out)[at] = r;
    else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(r);
    if (threadIdx.x == 0) a.lse[((int64_t)b * a.rows.Hq + head) * a.rows.n + j] = empty ? -INFINITY : fmaf(m, LN2, logf(l));
}

// The same by a warp per row, four rows a block, where a row has few pieces: the join is then
// bound by how many of its blocks find room beside the attention kernel's before that ends
// (64 ragged sequences up to 8192 tokens with a window of 1024, 2048 rows: 23 us with a block
// a row, 19.5 so).
template <typename A, int D, int NT, int DEEP>
__global__ void __launch_bounds__(128) kv_join_rows_kernel(A a, Shape sh, int warps, int rows)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int at_row = blockIdx.x * 4 + (threadIdx.x >> 5);
    const bool there = at_row < rows;
    const unsigned row_all = there ? (unsigned)at_row : 0u;
    const unsigned item = row_all / (unsigned)sh.rows, heads = sh.per_batch / sh.tiles;
    const int rr_all = (int)(row_all - item * sh.rows);
    const int b = (int)(item / heads), x = (int)(item - b * heads);   // x: (token, kv head)
    // as above: the lengths, and nothing else, before the wait
    static_assert(!Line<A>::NEXT_EARLY, "the next kernel starts behind the wait");
    int64_t all, before;
    count_blocks(a, b, all, before);
    all *= sh.per_batch;
    const Cuts cuts(all, warps, Line<A>::LEAST);
    const int nb = Line<A>::template blocks<true>(a, b);
    const int tile = rr_all / (NT * 8), row = rr_all % (NT * 8);
    const int h = x % a.pool.Hkv, j0 = x / a.pool.Hkv;
    const int i = (j0 * sh.tiles + tile) * a.pool.Hkv + h;
    const int64_t f = before * sh.per_batch + (int64_t)i * (nb + Line<A>::PAD);
    const int c0 = cuts.at(f), c1 = cuts.at(f + nb - 1);
    kv4_wait();
    kv4_trigger();
    if (!there || c0 == c1) return;
    const float *ws = static_cast<const float *>(a.ws);
    float m = -INFINITY, l = 0.f;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int c = c0; c <= c1; c += DEEP) {
        float pm[DEEP], pl[DEEP], v[DEEP][E], mn = m;
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            pm[u] = -INFINITY;
            pl[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
            if (c + u > c1) continue;
            const float *part = ws + (2 * (int64_t)(c + u) + (c + u == c0 ? 1 : 0)) * Part<D, NT>::FLOATS;
            pm[u] = part[row];
            pl[u] = part[8 * NT + row];
            if (E == 4) {
                const float4 w = *reinterpret_cast<const float4 *>(part + 16 * NT + row * D + lane * 4);
                v[u][0] = w.x, v[u][1] = w.y, v[u][E - 2] = w.z, v[u][E - 1] = w.w;
            } else {
                const float2 w = *reinterpret_cast<const float2 *>(part + 16 * NT + row * D + lane * 2);
                v[u][0] = w.x, v[u][1] = w.y;
            }
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u) mn = fmaxf(mn, pm[u]);
        const float fa = m == mn ? 1.f : ex2(m - mn);
        l *= fa;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= fa;
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            const float fu = pm[u] == mn ? 1.f : ex2(pm[u] - mn);
            l = fmaf(pl[u], fu, l);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(v[u][e], fu, o[e]);
        }
        m = mn;
    }
    const int j = j0 + rr_all / sh.group, head = h * sh.group + rr_all % sh.group;
    const bool empty = l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    const int64_t at = (((int64_t)b * a.rows.n + j) * a.rows.Hq + head) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        if (a.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at + e) = make_float2(o[e] * inv, o[e + 1] * inv);
        else *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + at + e) = tc::pack_bf16(o[e] * inv, o[e + 1] * inv);
    }
    if (lane == 0) a.lse[((int64_t)b * a.rows.Hq + head) * a.rows.n + j] = empty ? -INFINITY : fmaf(m, LN2, logf(l));
}

}  // namespace

}  // namespace cp
