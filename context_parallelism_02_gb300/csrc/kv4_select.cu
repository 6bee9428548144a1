// kv4_select.cu -- the pages that a query attends to, by a bound on its scores.
//
// A page's summary holds, per kv head, the smallest and largest value lo_d, hi_d of every
// element of its keys.  For any key k within them and a query row q
//   q.k <= sum_d max(q_d lo_d, q_d hi_d) = sum_d min(q_d, 0) lo_d + max(q_d, 0) hi_d,
// one product of length 2 D.  The summary is of the keys before quantisation, rounded to
// the nearest bf16, so the keys that attention reads may lie 2^-8 of the extremes and half
// a step of their groups outside: the bound ranks pages, it does not rule any out.
// A page's score is the largest bound of the query
// heads that share the kv head.  The n_sel best pages are kept, ties to the lower
// page, with the first and last pages of the sequence always among them.
//
// Scores: HBM-bound (4 D bytes per page and kv head), on mma.m16n8k16 with 16
// pages by 8 query heads, bf16 operands straight from memory, exact products,
// fp32 sums.
#include "kernels.h"
#include "kv4.cuh"

namespace cp {

namespace {

__device__ __forceinline__ void mma16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Both halves of a bf16 pair where their sign bit is (neg) or is not (!neg) set,
// 0 elsewhere.
__device__ __forceinline__ uint32_t half_line(uint32_t w, bool neg)
{
    uint32_t s;   // 0xffff in the halves whose sign is set: prmt that replicates the signs of bytes 1 and 3
    asm("prmt.b32 %0, %1, %1, 0xBB99;" : "=r"(s) : "r"(w));
    return neg ? w & s : w & ~s;
}

// A warp takes 16 pages of one (sequence, token, kv head) at a time; the page numbers
// of its next ones are on their way while it works.
template <int D>
__global__ void __launch_bounds__(128) kv4_score_kernel(Kv4SelectArgs a, int tiles, unsigned units)
{
    constexpr int NI = D / 16;   // 16-byte pieces of a summary row per lane
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    kv4_begin();
    const int Hkv = a.pool.Hkv, group = a.rows.Hq / Hkv, ps = a.pool.page_shift;
    const unsigned step = gridDim.x * 4;
    // a unit's place, and the page numbers of its tile (looked at below the length only)
    struct Place {
        unsigned item, bj;
        int tile, h, b, j, id[2];
    };
    auto place = [&](unsigned unit) {
        Place p;
        p.item = unit / (unsigned)tiles;
        p.bj = p.item / (unsigned)Hkv;
        p.tile = (int)(unit - p.item * tiles);
        p.h = (int)(p.item - p.bj * Hkv);
        p.b = (int)(p.bj / (unsigned)a.rows.n);
        p.j = (int)(p.bj - (unsigned)p.b * a.rows.n);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int lp = p.tile * 16 + r * 8 + g;
            p.id[r] = lp < a.pool.max_pages ? a.pool.pages[(int64_t)p.b * a.pool.max_pages + lp] : -1;
        }
        return p;
    };
    unsigned unit = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (unit >= units) return;
    Place p = place(unit);
    for (;;) {
        const int len = kv4_len(a.pool, p.b);
        const int lim = kv4_limit(a.rows, p.b, p.j, len);
        const int pages = (int)(((int64_t)lim + (1 << ps) - 1) >> ps);
        const bool any = p.tile * 16 < pages;
        uint4 w[2][NI];
        const uint4 *const q =
            reinterpret_cast<const uint4 *>(a.q + ((int64_t)p.bj * a.rows.Hq + p.h * group + min(g, group - 1)) * D);
        uint4 q0[NI / 2];
        if (any) {
#pragma unroll
            for (int i = 0; i < NI / 2; ++i) q0[i] = q[i * 4 + c];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int lp = p.tile * 16 + r * 8 + g;
                int id = p.id[r];
                if (lp >= pages) {
                    id = -1;
                } else if (id < 0 || id >= a.pool.n_pages) {
                    kv4_report(a.pool.err);
                    id = -1;
                }
                const uint4 *s = reinterpret_cast<const uint4 *>(a.summary + ((int64_t)(id < 0 ? 0 : id) * Hkv + p.h) * 2 * D);
#pragma unroll
                for (int i = 0; i < NI; ++i) w[r][i] = id >= 0 ? s[i * 4 + c] : make_uint4(0, 0, 0, 0);
            }
        }
        const Place now = p;
        unit += step;
        const bool more = unit < units;
        if (more) p = place(unit);
        if (any) {
            float best[2] = {-INFINITY, -INFINITY};
            bool nan[2] = {false, false};
            for (int h0 = 0; h0 < group; h0 += 8) {
                // heads past the group repeat its last one: their columns are not looked at
                const uint4 *qh = q + (int64_t)(min(h0 + g, group - 1) - min(g, group - 1)) * (D / 8);
                float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};   // two chains
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const bool neg = i < NI / 2;
                    const int x4 = neg ? i : i - NI / 2;
                    const uint4 x = h0 == 0 ? q0[x4] : qh[x4 * 4 + c];
                    mma16816_bf16(acc, w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y, half_line(x.x, neg), half_line(x.y, neg));
                    mma16816_bf16(acc2, w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w, half_line(x.z, neg), half_line(x.w, neg));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (h0 + 2 * c + (e & 1) < group) {
                        const float sum = acc[e] + acc2[e];
                        best[e >> 1] = fmaxf(best[e >> 1], sum);
                        nan[e >> 1] |= isnan(sum);
                    }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float v = nan[r] ? INFINITY : best[r];   // a page whose bound is not a number comes first
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                const int lp = now.tile * 16 + r * 8 + g;
                if (c == 0 && lp < pages) a.scores[(int64_t)now.item * a.pool.max_pages + lp] = v;
            }
        }
        if (!more) return;
    }
}

// A score as an unsigned key of the same order; pages that are always kept
// above every score.
__device__ __forceinline__ uint32_t page_key(const Kv4SelectArgs &a, const float *scores, int lp, int pages)
{
    if (lp < a.keep_first || lp >= pages - a.keep_last) return 0xffffffffu;
    const float f = scores[lp] + 0.f;   // -0 counts as 0
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int SEL_THREADS = 256;   // 2048 pages: 9.3 us for the two kernels, with 512 9.9

// Sum over the block; red has two halves that calls use in turn, so that one
// barrier a call is enough.
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t (*red)[SEL_THREADS / 32], int &turn)
{
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const uint32_t s = __reduce_add_sync(0xffffffffu, lane < SEL_THREADS / 32 ? red[turn][lane] : 0u);
    turn ^= 1;
    return s;
}

// Two sums behind one barrier.
__device__ __forceinline__ void block_sum2(uint32_t &v, uint32_t &w, uint32_t (*red)[SEL_THREADS / 32],
                                           uint32_t (*red2)[SEL_THREADS / 32], int &turn)
{
    v = __reduce_add_sync(0xffffffffu, v);
    w = __reduce_add_sync(0xffffffffu, w);
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[turn][threadIdx.x >> 5] = v, red2[turn][threadIdx.x >> 5] = w;
    __syncthreads();
    v = __reduce_add_sync(0xffffffffu, lane < SEL_THREADS / 32 ? red[turn][lane] : 0u);
    w = __reduce_add_sync(0xffffffffu, lane < SEL_THREADS / 32 ? red2[turn][lane] : 0u);
    turn ^= 1;
}

// Sum over the threads before this one.
__device__ __forceinline__ uint32_t block_before(uint32_t v, uint32_t (*red)[SEL_THREADS / 32], int &turn)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += w;
    }
    if (lane == 31) red[turn][warp] = upto;
    __syncthreads();
    const uint32_t s = __reduce_add_sync(0xffffffffu, lane < warp ? red[turn][lane] : 0u);
    turn ^= 1;
    return s + upto - v;
}

// The n_sel-th largest key of a row's pages, two bits at a time from the top, then
// the pages above it and the first of those equal to it, in page order.  A thread has
// up to K neighbouring pages in registers; K = 0: any number, and the scores are read
// again for every step.
template <int K>
__device__ __forceinline__ void take_top(const Kv4SelectArgs &a, const float *scores, int32_t *sel, int pages,
                                         uint32_t (*red)[SEL_THREADS / 32], uint32_t (*red2)[SEL_THREADS / 32])
{
    int turn = 0;
    const int each = (pages + SEL_THREADS - 1) / SEL_THREADS;   // at most K, unless K = 0
    const int first = min((int)threadIdx.x * each, pages), mine = min(each, pages - first);
    uint32_t key[K > 0 ? K : 1];
#pragma unroll
    for (int i = 0; i < K; ++i) key[i] = i < mine ? page_key(a, scores, first + i, pages) : 0u;
    // number of keys at or above a bound > 0 (no page has key 0: -inf's is 0x007fffff)
    auto at_least = [&](uint32_t bound) {
        uint32_t n = 0;
        if (K > 0) {
#pragma unroll
            for (int i = 0; i < K; ++i) n += key[i] >= bound;
        } else {
            for (int i = 0; i < mine; ++i) n += page_key(a, scores, first + i, pages) >= bound;
        }
        return n;
    };
    const uint32_t want = (uint32_t)a.n_sel;
    uint32_t thr = 0, have = pages;   // pages at or above thr: once that is what is wanted, the bits below do not matter
    if (K > 0) {   // fewer than 2^16 pages: three counts in two sums of halves
        for (int bit = 30; bit >= 0 && have != want; bit -= 2) {
            uint32_t s12 = at_least(thr | 1u << bit) | at_least(thr | 2u << bit) << 16, s3 = at_least(thr | 3u << bit);
            block_sum2(s12, s3, red, red2, turn);
            if (s3 >= want) thr |= 3u << bit, have = s3;
            else if (s12 >> 16 >= want) thr |= 2u << bit, have = s12 >> 16;
            else if ((s12 & 0xffffu) >= want) thr |= 1u << bit, have = s12 & 0xffffu;
        }
    } else {
        for (int bit = 31; bit >= 0 && have != want; --bit) {
            const uint32_t s = block_sum(at_least(thr | 1u << bit), red, turn);
            if (s >= want) thr |= 1u << bit, have = s;
        }
    }
    // with as many pages at or above thr as are wanted, all of them count as above
    if (have == want) --thr;
    const uint32_t gt = thr == 0xffffffffu ? 0u : at_least(thr + 1), eq = have == want ? 0u : at_least(thr) - gt;
    const uint32_t ties = want - block_sum(gt, red, turn);   // pages equal to the threshold that are taken
    uint32_t seen = block_before(eq, red, turn);             // ... that come before this thread's
    uint32_t at = block_before(gt, red, turn) + min(seen, ties);
    auto put = [&](uint32_t k, int page) {
        if (k > thr) sel[at++] = page;
        else if (k == thr && seen++ < ties) sel[at++] = page;
    };
    if (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < mine) put(key[i], first + i);
    } else {
        for (int i = 0; i < mine; ++i) put(page_key(a, scores, first + i, pages), first + i);
    }
}

// One block per (sequence, token, kv head).
__global__ void __launch_bounds__(SEL_THREADS) kv4_top_kernel(Kv4SelectArgs a)
{
    __shared__ uint32_t red[2][SEL_THREADS / 32], red2[2][SEL_THREADS / 32];
    kv4_begin();
    const unsigned item = blockIdx.x, bj = item / (unsigned)a.pool.Hkv;
    const int b = (int)(bj / (unsigned)a.rows.n), j = (int)(bj - (unsigned)b * a.rows.n);
    const int len = kv4_len(a.pool, b);
    const int lim = kv4_limit(a.rows, b, j, len);
    const int ps = a.pool.page_shift;
    const int pages = (int)(((int64_t)lim + (1 << ps) - 1) >> ps);
    const float *scores = a.scores + (int64_t)item * a.pool.max_pages;
    int32_t *sel = a.sel + (int64_t)item * a.n_sel;
    if (pages <= a.n_sel) {
        for (int i = threadIdx.x; i < a.n_sel; i += SEL_THREADS) sel[i] = i < pages ? i : -1;
        return;
    }
    // with two keys a thread a step is its barrier, with 32 its comparisons
    if (pages <= 2 * SEL_THREADS) take_top<2>(a, scores, sel, pages, red, red2);
    else if (pages <= 8 * SEL_THREADS) take_top<8>(a, scores, sel, pages, red, red2);
    else if (pages <= 32 * SEL_THREADS) take_top<32>(a, scores, sel, pages, red, red2);
    else take_top<0>(a, scores, sel, pages, red, red2);
}

}  // namespace

int launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st)
{
    const int64_t items = (int64_t)a.rows.B * a.rows.n * a.pool.Hkv;
    const int tiles = (a.pool.max_pages + 15) / 16;
    const int64_t warps = items * tiles;
    if (items > 0x7fffffffLL || warps > 0x3fffffffLL) return CP_EUNSUPPORTED;
    // four waves of blocks (16 sequences of up to 1024 pages: both kernels 16.0 us; one
    // wave, whose warps loop more, 17.9: ragged lengths leave some with little to do)
    const int64_t grid = min((warps + 3) / 4, (int64_t)sm_count() * 16);
    if (grid > 0) {
        const cudaError_t rc =
            D == 64 ? kv4_launch(kv4_score_kernel<64>, (unsigned)grid, 128, 0, st, a, tiles, (unsigned)warps)
                    : kv4_launch(kv4_score_kernel<128>, (unsigned)grid, 128, 0, st, a, tiles, (unsigned)warps);
        if (rc != cudaSuccess) return CP_ECUDA;
    }
    return kv4_launch(kv4_top_kernel, (unsigned)items, SEL_THREADS, 0, st, a) == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace cp
