// kv4_select.cu -- the pages that a query attends to, by a bound on its scores.
//
// A page's summary holds, per kv head, the smallest and largest value of every
// element of its keys.  For any key k of the page and a query row q
//   q.k <= sum_d max(q_d lo_d, q_d hi_d) = sum_d min(q_d, 0) lo_d + max(q_d, 0) hi_d,
// one product of length 2 D; a page's score is the largest bound of the query
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
    const uint32_t s = ((w >> 15) & 0x00010001u) * 0xffffu;
    return neg ? w & s : w & ~s;
}

// One warp per 16 pages of one (sequence, token, kv head).
template <int D>
__global__ void __launch_bounds__(128) kv4_score_kernel(Kv4SelectArgs a, int tiles, int64_t warps)
{
    constexpr int NI = D / 16;   // 16-byte pieces of a summary row per lane
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (wid >= warps) return;
    const int Hkv = a.pool.Hkv, group = a.rows.Hq / Hkv;
    const int tile = (int)(wid % tiles);
    const int64_t item = wid / tiles;
    const int h = (int)(item % Hkv);
    const int64_t bj = item / Hkv;
    const int j = (int)(bj % a.rows.n), b = (int)(bj / a.rows.n);
    const int len = kv4_len(a.pool, b);
    const int lim = kv4_limit(a.rows, b, j, len);
    const int ps = a.pool.page_shift;
    const int pages = (int)(((int64_t)lim + (1 << ps) - 1) >> ps);
    if (tile * 16 >= pages) return;
    uint4 w[2][NI];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int lp = tile * 16 + r * 8 + g;
        const int id = lp < pages ? kv4_page(a.pool, b, lp) : -1;
        const uint4 *p = reinterpret_cast<const uint4 *>(a.summary + ((int64_t)(id < 0 ? 0 : id) * Hkv + h) * 2 * D);
#pragma unroll
        for (int i = 0; i < NI; ++i) w[r][i] = id >= 0 ? __ldg(p + i * 4 + c) : make_uint4(0, 0, 0, 0);
    }
    float best[2] = {-INFINITY, -INFINITY};
    bool nan[2] = {false, false};
    for (int h0 = 0; h0 < group; h0 += 8) {
        const bool on = h0 + g < group;
        const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (bj * a.rows.Hq + h * group + (on ? h0 + g : 0)) * D);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool neg = i < NI / 2;
            const uint4 x = __ldg(q + (neg ? i : i - NI / 2) * 4 + c);
            mma16816_bf16(acc, w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y, half_line(x.x, neg), half_line(x.y, neg));
            mma16816_bf16(acc, w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w, half_line(x.z, neg), half_line(x.w, neg));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (h0 + 2 * c + (e & 1) < group) {
                best[e >> 1] = fmaxf(best[e >> 1], acc[e]);
                nan[e >> 1] |= isnan(acc[e]);
            }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float v = nan[r] ? INFINITY : best[r];   // a page whose bound is not a number comes first
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        const int lp = tile * 16 + r * 8 + g;
        if (c == 0 && lp < pages) a.scores[item * a.pool.max_pages + lp] = v;
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

constexpr int SEL_THREADS = 256;

__device__ __forceinline__ int block_sum(int v, int *red)
{
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < SEL_THREADS / 32; ++w) s += red[w];
    return s;
}

// One block per (sequence, token, kv head): the n_sel-th largest key bit by bit,
// then the pages above it and the first of those equal to it, in page order.
__global__ void __launch_bounds__(SEL_THREADS) kv4_top_kernel(Kv4SelectArgs a)
{
    __shared__ int red[SEL_THREADS / 32];
    const int64_t item = blockIdx.x;
    const int64_t bj = item / a.pool.Hkv;
    const int j = (int)(bj % a.rows.n), b = (int)(bj / a.rows.n);
    const int len = kv4_len(a.pool, b);
    const int lim = kv4_limit(a.rows, b, j, len);
    const int ps = a.pool.page_shift;
    const int pages = (int)(((int64_t)lim + (1 << ps) - 1) >> ps);
    const float *scores = a.scores + item * a.pool.max_pages;
    int32_t *sel = a.sel + item * a.n_sel;
    if (pages <= a.n_sel) {
        for (int i = threadIdx.x; i < a.n_sel; i += SEL_THREADS) sel[i] = i < pages ? i : -1;
        return;
    }
    uint32_t thr = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = thr | 1u << bit;
        int n = 0;
        for (int i = threadIdx.x; i < pages; i += SEL_THREADS) n += page_key(a, scores, i, pages) >= cand;
        if (block_sum(n, red) >= a.n_sel) thr = cand;
    }
    int above = 0;
    for (int i = threadIdx.x; i < pages; i += SEL_THREADS) above += page_key(a, scores, i, pages) > thr;
    const int ties = a.n_sel - block_sum(above, red);   // pages equal to the threshold that are taken
    int done = 0, seen = 0;                             // pages written, ties met, before this stretch
    for (int i0 = 0; i0 < pages; i0 += SEL_THREADS) {
        const int i = i0 + threadIdx.x;
        const uint32_t k = i < pages ? page_key(a, scores, i, pages) : 0u;
        const bool eq = i < pages && k == thr, gt = i < pages && k > thr;
        // exclusive counts over the block
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const unsigned be = __ballot_sync(0xffffffffu, eq), bg = __ballot_sync(0xffffffffu, gt);
        __syncthreads();
        if (lane == 0) red[warp] = __popc(be) << 16 | __popc(bg);
        __syncthreads();
        int pe = 0, pg = 0, te = 0, tg = 0;
        for (int w = 0; w < SEL_THREADS / 32; ++w) {
            const int e = red[w] >> 16, q = red[w] & 0xffff;
            if (w < warp) pe += e, pg += q;
            te += e, tg += q;
        }
        const unsigned below = (1u << lane) - 1u;
        const int my_e = seen + pe + __popc(be & below);   // ties before this page
        const int my_g = pg + __popc(bg & below);
        const int taken_e = min(my_e, ties) - min(seen, ties);
        if (gt || (eq && my_e < ties)) sel[done + my_g + taken_e] = i;
        done += tg + min(seen + te, ties) - min(seen, ties);
        seen += te;
    }
}

}  // namespace

int launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st)
{
    const int64_t items = (int64_t)a.rows.B * a.rows.n * a.pool.Hkv;
    const int tiles = (a.pool.max_pages + 15) / 16;
    const int64_t warps = items * tiles;
    const int64_t grid = (warps + 3) / 4;
    if (items > 0x7fffffffLL || grid > 0x7fffffffLL) return CP_EUNSUPPORTED;
    if (D == 64) kv4_score_kernel<64><<<(unsigned)grid, 128, 0, st>>>(a, tiles, warps);
    else kv4_score_kernel<128><<<(unsigned)grid, 128, 0, st>>>(a, tiles, warps);
    if (cudaGetLastError() != cudaSuccess) return CP_ECUDA;
    kv4_top_kernel<<<(unsigned)items, SEL_THREADS, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace cp
