// kv8_attn.cu -- attention of a few query tokens over the paged 8-bit cache, whole or
// with a sliding window and sinks, and the weight that every cached slot got.
//
//   s_ij = scale q_i . k_j over the slots j that row i sees,
//   lse_i = ln sum_j e^{s_ij},   out_i = sum_j e^{s_ij - lse_i} v_j;
//   a row that sees nothing: (0, -inf).   mass_j += sum_i e^{s_ij - lse_i}.
//
// HBM-bound for few query rows: a token and kv head is 2 D bytes and a block's two scales,
// read once for all rows of the tile.  The schedule is kv_line.cuh's; blocks of 16 rows
// arrive by TMA in the swizzled order that makes the reads below free of bank conflicts.
// The work of a block is two products on mma.m16n8k16 with the cache as the A operand,
// S^T = K q^T and O^T += V^T P^T: 16 tokens (or 16 d) by 8 query rows, so that the few
// rows of a decode step fill the narrow side of the instruction, and a lane turns exactly
// the codes that it feeds to the tensor core into fp16 (exact, one conversion a pair).
//
// Scores: q is scaled per row by a power of two so that its largest element comes to 2^14:
// bf16's 8 bits fit fp16 down to 2^-31 of it, and the products are exact; the block's K
// scale and the row's multiply the fp32 sums.
// V's codes are exact in fp16, and a block's V scale 2^e goes into its weights: they are
// P' = 2^(x + e - m), x the score in log2 units and m a reference 7 to 15 powers of two
// below the largest x + e so far, so that O sums codes in units of 2^m and what is rounded
// (P' to fp16: 2^-11 of itself, or 2^-32 of the largest) is the product of a weight and
// its block's scale, whichever of the two is small.  The row sums take P' 2^-e, unrounded.
//
// 16 x 32768 tokens, 32 heads on 8, D = 128: 160.6 us, the rate of a copy; 64 ragged sequences
// up to 8192 under a window of 1024 and 4 sinks 19.6 (47 MB: starts and the join); one of 512
// tokens 7.0 (four dependent loads); 8 x 16384, 16 heads on 8, D = 64 27.7 for one token each,
// 43.2 for four with the weights added up.
#include <atomic>

#include <cuda.h>

#include "kernels.h"
#include "kv8.cuh"
#include "kv_line.cuh"
#include "tc_helpers.cuh"

namespace cp {

// Blocks of one item: with a window those of the sinks and those that some row's window
// reaches; `skip` blocks lie between.  The rows' limits are len - (n - 1) ... len (causal),
// or in vis, on the device: then every block counts.
struct Kv8Span {
    int blocks, sinks, skip;
    __device__ __forceinline__ Kv8Span(const Kv8AttnArgs &a, int len)
    {
        const int all = len > 0 ? (len - 1) / KV8_BLOCK + 1 : 1;
        blocks = all;
        sinks = skip = 0;
        if (a.window > 0 && !a.rows.vis) {
            const int64_t first = (int64_t)len - (a.rows.causal ? a.rows.n - 1 : 0) - a.window;   // of the first row
            const int from = first > 0 ? (int)(first / KV8_BLOCK) : 0;
            sinks = (int)(((int64_t)a.sinks + KV8_BLOCK - 1) / KV8_BLOCK);
            if (sinks < from) {
                skip = from - sinks;
                blocks = all - skip;
            }
        }
    }
    // block number of the item's t-th
    __device__ __forceinline__ int block(int t) const { return t < sinks ? t : t + skip; }
};

template <>
struct Line<Kv8AttnArgs> {
    static constexpr int PAD = 8;
    static constexpr int LEAST = 2;   // a stage
    static constexpr bool NEXT_EARLY = false;
    template <bool EARLY>
    __device__ __forceinline__ static int blocks(const Kv8AttnArgs &a, int b)
    {
        return Kv8Span(a, kv4_len<EARLY>(a.pool, b)).blocks;
    }
};

namespace {

constexpr int WARPS = 4;
constexpr int PAD = Line<Kv8AttnArgs>::PAD, LEAST = Line<Kv8AttnArgs>::LEAST;
// Rows of warps' parts in the workspace (twice): of all warps that run at once.  16 rows of 64
// elements need more than MAX_ROWS: with two blocks on most SMs and three on some a step of 5
// tokens, 20 rows a kv head, over 64 x 1024 took 55 us, with room for three on all 45.
__host__ __device__ constexpr int part_rows(int D) { return D == 64 ? MAX_ROWS / 2 * 3 : MAX_ROWS; }
static_assert(part_rows(64) / 8 < MAX_STRETCHES && part_rows(128) / 8 < MAX_STRETCHES, "a warp's part has 8 rows at least");
constexpr int NB = 2;              // blocks of a stage, taken together
constexpr int STAGES = 2;          // of a warp's ring

// Query rows of one tile, as B operands, and what goes with a row.  Lane (g, c) =
// (lane / 4, lane % 4) holds row 8 t + g's share in q, the elements D / 4 c + 4 s + {0,1}
// and {2,3} for k-step s; the accumulators' columns are rows 8 t + 2c and 8 t + 2c + 1.
template <int D, int NT>
struct Rows {
    uint32_t q[NT][D / 16][2];
    float to_log2[NT][2];      // score -> log2 units, for the lane's two columns
    int limit[NT][2], low[NT][2];   // slots that the column's row sees: [low, limit) and the sinks
    int min_limit, max_limit;  // over the tile
    int min_low, max_low;
};

// Running state of a warp: m in log2 units, l per lane (its own tokens), O^T accumulators.
// O's tile i, row g (and g + 8): d = D / 8 g + 2 i (and one more).
template <int D, int NT>
struct State {
    float m[NT][2], l[NT][2];
    float o[NT][D / 16][4];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
        }
    }
};

// A lane's share of the rows as they are in memory: D / 4 elements of a row.
template <int D, int NT>
struct RawRows {
    uint4 w[NT][D / 32];
};

template <int D, int NT>
__device__ __forceinline__ void fetch_rows(const Kv8AttnArgs &a, const Shape &sh, const Item &it, RawRows<D, NT> &raw)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = (it.tile * NT + t) * 8 + g;
        const bool on = row < sh.rows;
        const int j = on ? row / sh.group : 0;
        const int head = it.h * sh.group + (on ? row % sh.group : 0);
        const uint4 *p = reinterpret_cast<const uint4 *>(a.q + (((int64_t)it.b * a.rows.n + j) * a.rows.Hq + head) * D);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw.w[t][i] = on ? p[c * (D / 32) + i] : make_uint4(0, 0, 0, 0);
    }
}

template <int D, int NT>
__device__ __forceinline__ void make_rows(const Kv8AttnArgs &a, const Shape &sh, const Item &it, int len,
                                          const RawRows<D, NT> &raw, Rows<D, NT> &r)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    int lo = 0x7fffffff, hi = 0, lo_low = 0x7fffffff, hi_low = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = (it.tile * NT + t) * 8 + g;
        const bool on = row < sh.rows;
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t x[4] = {raw.w[t][i].x, raw.w[t][i].y, raw.w[t][i].z, raw.w[t][i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xffff0000u))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // q 2^s has its largest magnitude in [2^14, 2^15)
        int s = 0;
        if (top > 0.f && top < INFINITY) s = 14 - ilogbf(top);
        s = s > 120 ? 120 : s < -120 ? -120 : s;
        const float up = __int_as_float((127 + s) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t x[4] = {raw.w[t][i].x, raw.w[t][i].y, raw.w[t][i].z, raw.w[t][i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)   // elements 8 i + 2 e, 8 i + 2 e + 1 of the lane's share
                r.q[t][2 * i + (e >> 1)][e & 1] =
                    h2(__floats2half2_rn(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xffff0000u) * up));
        }
        // with an infinity in the row all visible scores could be -infinity, which the end would
        // take for a row that sees nothing: NaN (which fp16 elements that are NaN bring by themselves)
        const float back = top < INFINITY ? a.scale * LOG2E / up : __int_as_float(0x7fffffff);
        const int lim = on ? kv4_limit(a.rows, it.b, row / sh.group, len) : 0;
        const int low = a.window > 0 && on ? max(lim - a.window, 0) : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            r.to_log2[t][e] = __shfl_sync(0xffffffffu, back, (2 * c + e) * 4);
            r.limit[t][e] = __shfl_sync(0xffffffffu, lim, (2 * c + e) * 4);
            r.low[t][e] = __shfl_sync(0xffffffffu, low, (2 * c + e) * 4);
        }
        lo = min(lo, on ? lim : 0x7fffffff);
        hi = max(hi, lim);
        lo_low = min(lo_low, on ? low : 0x7fffffff);
        hi_low = max(hi_low, low);
    }
    r.min_limit = __reduce_min_sync(0xffffffffu, lo);
    r.max_limit = __reduce_max_sync(0xffffffffu, hi);
    r.min_low = __reduce_min_sync(0xffffffffu, lo_low);
    r.max_low = __reduce_max_sync(0xffffffffu, hi_low);
}

// 16 bytes at chunk ch of row r of a tile of 16 rows of D bytes, in TMA's swizzled order
// (of 128 bytes for D = 128, of 64 for D = 64): the chunk's bits are xored with the row's.
template <int D>
__device__ __forceinline__ uint4 tile_chunk(const uint8_t *tile, int r, int ch)
{
    const int x = D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3);
    return *reinterpret_cast<const uint4 *>(tile + r * D + x * 16);
}

// Scores of one block before scaling: x[t][0..1] token g, x[t][2..3] token g + 8.
template <int D, int NT>
__device__ __forceinline__ void block_scores(const uint8_t *tile, const Rows<D, NT> &r, float (&x)[NT][4])
{
    constexpr int CH = D / 64;   // 16-byte chunks of a lane and row
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint4 k[2][CH];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < CH; ++i) k[hf][i] = tile_chunk<D>(tile, g + 8 * hf, c * CH + i);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const uint4 &ka = k[0][s >> 2], &kb = k[1][s >> 2];
        const uint32_t wa = (s & 3) == 0 ? ka.x : (s & 3) == 1 ? ka.y : (s & 3) == 2 ? ka.z : ka.w;
        const uint32_t wb = (s & 3) == 0 ? kb.x : (s & 3) == 1 ? kb.y : (s & 3) == 2 ? kb.z : kb.w;
        const uint32_t a0 = kv8_halves(wa & 0xffffu), a2 = kv8_halves(wa >> 16);
        const uint32_t a1 = kv8_halves(wb & 0xffffu), a3 = kv8_halves(wb >> 16);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (s == 0) mma16816_zero(x[t], a0, a1, a2, a3, r.q[t][s][0], r.q[t][s][1]);
            else mma16816(x[t], a0, a1, a2, a3, r.q[t][s][0], r.q[t][s][1]);
        }
    }
}

// The references m lie this far below the largest score when they are raised, and are
// raised where a score passes them by more than 15: 2^15 is an fp16.
constexpr float BELOW = 7.f, LAG = 15.f;

template <int D, int NT>
__device__ __forceinline__ void raise_max(const float (&x)[NB][NT][4], State<D, NT> &s)
{
    bool high = false;
    float top[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = fmaxf(x[0][t][e], x[0][t][e + 2]);
#pragma unroll
            for (int i = 1; i < NB; ++i) v = fmaxf(v, fmaxf(x[i][t][e], x[i][t][e + 2]));
            top[t][e] = v;
            // the difference, exact for neighbours: m + 15 rounds up to m + 16 where floats lie 16 apart
            high |= v - s.m[t][e] > LAG;
        }
    if (!__any_sync(0xffffffffu, high)) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = top[t][e];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            const float m = fmaxf(s.m[t][e], v - BELOW);
            const float f = m == -INFINITY ? 1.f : ex2(s.m[t][e] - m);
            s.m[t][e] = m;
            s.l[t][e] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) s.o[t][i][e] *= f, s.o[t][i][e + 2] *= f;
        }
}

// Whether a word of codes holds NaN (magnitude bits all ones), as a bit at each byte's top.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// O^T += V^T P^T for one block, p the weights as B operands.  CUT: some row does not see
// all of the block's tokens; see: what the lane's two columns see, live: what any row of
// the tile sees.  A token that no row sees may hold anything, and one that only some rows
// see may hold NaN, which 0 times would carry to the others: both count as 0, and the rows
// that do see a NaN get it afterwards.
template <int D, int NT, bool CUT>
__device__ __forceinline__ void block_values(const uint8_t *tile, const uint32_t (&see)[NT][2], uint32_t live,
                                             const uint32_t (&p)[NT][2], State<D, NT> &s)
{
    constexpr int WORDS = D / 32;   // of a lane and token: D / 8 elements
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint32_t w[4][WORDS];           // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 2 * c + (i & 1) + (i >> 1) * 8;
        if (D == 128) {
            const uint4 v = tile_chunk<D>(tile, r, g);
            w[i][0] = v.x, w[i][1] = v.y, w[i][WORDS - 2] = v.z, w[i][WORDS - 1] = v.w;
        } else {
            const int x = (g >> 1) ^ ((r >> 1) & 3);
            const uint2 v = *reinterpret_cast<const uint2 *>(tile + r * D + x * 16 + (g & 1) * 8);
            w[i][0] = v.x, w[i][WORDS - 1] = v.y;
        }
    }
    uint32_t bad = 0;               // CUT: tokens with a NaN, any d of the lane
    if (CUT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * c + (i & 1) + (i >> 1) * 8;
#pragma unroll
            for (int j = 0; j < WORDS; ++j) {
                if (!(live >> r & 1u)) w[i][j] = 0;
                if (nan_bytes(w[i][j])) bad |= 1u << r;
            }
        }
    }
    const bool any_bad = CUT && __any_sync(0xffffffffu, bad != 0);
    uint32_t mark[D / 8] = {};      // per d of the lane: tokens with a NaN there
    if (any_bad) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * c + (i & 1) + (i >> 1) * 8;
#pragma unroll
            for (int j = 0; j < WORDS; ++j) {
                const uint32_t n = nan_bytes(w[i][j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n >> (8 * e + 7) & 1u) {
                        mark[4 * j + e] |= 1u << r;
                        w[i][j] &= ~(0xffu << (8 * e));
                    }
            }
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
            mark[d] |= __shfl_xor_sync(0xffffffffu, mark[d], 1);
            mark[d] |= __shfl_xor_sync(0xffffffffu, mark[d], 2);
        }
    }
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
        // bytes (token 2c, token 2c + 1) of elements 0, 1 and 2, 3 of the word, and the same 8 tokens on
        const uint32_t x01 = __byte_perm(w[0][j], w[1][j], 0x5140), x23 = __byte_perm(w[0][j], w[1][j], 0x7362);
        const uint32_t y01 = __byte_perm(w[2][j], w[3][j], 0x5140), y23 = __byte_perm(w[2][j], w[3][j], 0x7362);
        const uint32_t f[2][4] = {{kv8_halves(x01 & 0xffffu), kv8_halves(x01 >> 16), kv8_halves(y01 & 0xffffu), kv8_halves(y01 >> 16)},
                                  {kv8_halves(x23 & 0xffffu), kv8_halves(x23 >> 16), kv8_halves(y23 & 0xffffu), kv8_halves(y23 >> 16)}};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) mma16816(s.o[t][2 * j + i], f[i][0], f[i][1], f[i][2], f[i][3], p[t][0], p[t][1]);
    }
    if (any_bad) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    if (mark[d] & see[t][e]) s.o[t][d >> 1][e + 2 * (d & 1)] = __int_as_float(0x7fffffff);
    }
}

// The scales that an append or an eviction writes lie between these.
constexpr float MIN_SCALE = 1.f / (1ull << -KV8_E_MIN), MAX_SCALE = (float)(1ull << KV8_E_MAX);

// What goes with a block in the ring.
struct Meta {
    int slot;            // its first slot, or NO_SLOT
    float k, v;          // its scales
};

// The columns' visible tokens of the block that begins at slot.
template <int D, int NT>
__device__ __forceinline__ void visible_tokens(const Rows<D, NT> &r, int slot, int sinks, uint32_t (&see)[NT][2])
{
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            see[t][e] = slot == NO_SLOT ? 0u
                                        : visible_bits(0, min(r.limit[t][e] - slot, KV8_BLOCK), r.low[t][e] - slot, sinks - slot) & 0xffffu;
}

// Rows of a token's scores: those of its kv head, rounded up so that they are read by fours.
__host__ __device__ __forceinline__ int64_t score_rows(int64_t rows) { return (rows + 3) / 4 * 4; }

// A stage: NB blocks of 16 tokens for the warp's state.  scores: those of the item's kv head,
// [slot][rows], or null.
template <int D, int NT>
__device__ __forceinline__ void blocks_step(const uint8_t *stage, const Meta (&mt)[NB], const Rows<D, NT> &r, int sinks,
                                            float *scores, int rows, int tile_row, State<D, NT> &s)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float x[NB][NT][4], ev[NB];
    bool cut[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        block_scores<D, NT>(stage + i * 32 * D, r, x[i]);
        cut[i] = mt[i].slot > r.min_limit - KV8_BLOCK || (mt[i].slot < r.max_low && mt[i].slot + KV8_BLOCK > sinks);
        ev[i] = (float)((int)(__float_as_uint(mt[i].v) >> 23) - 127);
        // rounded here and not fused with the subtraction of m, which is one of these
        // products: a difference is then at most LAG however large the scores are
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][t][e] = __fmul_rn(x[i][t][e], r.to_log2[t][e & 1] * mt[i].k);
    }
    uint32_t see[NB][NT][2];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        if (!cut[i]) continue;
        visible_tokens<D, NT>(r, mt[i].slot, sinks, see[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(see[i][t][e & 1] >> (g + (e >> 1) * 8) & 1u)) x[i][t][e] = -INFINITY;
    }
    if (scores) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (mt[i].slot == NO_SLOT) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int row = tile_row + 8 * t + 2 * c;
                    if (row < rows)
                        *reinterpret_cast<float2 *>(scores + ((int64_t)mt[i].slot + g + hf * 8) * rows + row) =
                            make_float2(x[i][t][2 * hf], x[i][t][2 * hf + 1]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][t][e] = __fadd_rn(x[i][t][e], ev[i]);
    raise_max<D, NT>(x, s);
    uint32_t p[NB][NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) base[e] = s.m[t][e] == -INFINITY ? 0.f : -s.m[t][e];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float w[4];
            const float inv = __uint_as_float((254u << 23) - __float_as_uint(mt[i].v));   // 2^-e
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = ex2(__fadd_rn(x[i][t][e], base[e & 1]));
                s.l[t][e & 1] = fmaf(w[e], inv, s.l[t][e & 1]);
            }
            p[i][t][0] = movmatrix(h2(__floats2half2_rn(w[0], w[1])));
            p[i][t][1] = movmatrix(h2(__floats2half2_rn(w[2], w[3])));
        }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const uint8_t *v = stage + i * 32 * D + 16 * D;
        if (!cut[i]) {
            block_values<D, NT, false>(v, see[i], 0xffffu, p[i], s);
            continue;
        }
        uint32_t live = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) live |= see[i][t][0] | see[i][t][1];
        live = __reduce_or_sync(0xffffffffu, live);
        if (live) block_values<D, NT, true>(v, see[i], live, p[i], s);
    }
}

template <int D, int W>
struct Smem {
    alignas(1024) uint8_t ring[W][STAGES][NB][32 * D];   // K's 16 rows, then V's
    uint64_t full[W][STAGES];
    uint64_t hold;                       // completed by nobody: what the failure path is tested with
    Meta meta[W][STAGES][NB];
    Walk ahead[W];                       // the piece that a warp's copies are issued for
    int abort, never;
};

// 16 rows of a (page, kv head, K or V) plane by TMA.
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int row, int plane, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(0), "r"(row), "r"(plane), "l"(policy)
        : "memory");
}

// ALONE: a block per item, its W warps share the item's blocks evenly and join in
// shared memory, and there is no second kernel (short tables); else kv_line.cuh's schedule.
template <int D, int NT, int W, bool ALONE>
__global__ void __launch_bounds__(W * 32)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap map, Kv8AttnArgs a, Shape sh, int warps)
{
    extern __shared__ __align__(1024) uint8_t dyn[];
    Smem<D, W> &sm = *reinterpret_cast<Smem<D, W> *>(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    if (smem_u32(dyn) & 1023u) {   // the swizzle goes by the address
        if (threadIdx.x == 0) atomicCAS(a.pool.err, 0u, ERRW_SMEM_ALIGN);
        return;
    }
    if (lane < STAGES) mbar_init(smem_u32(&sm.full[warp][lane]), NB);
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sm.hold), 1);
        sm.abort = sm.never = 0;
    }
    fence_mbar_init();
    // not kv4_begin: the join reads the lengths before its own wait, so it may start only
    // when every block here is past this one
    kv4_wait();
    kv4_trigger();
    {   // what the chain of loads below will need, on its way to L2
        const int64_t line = ((int64_t)blockIdx.x * (W * 32) + threadIdx.x) * 128;
        prefetch(a.pool.pages, line, (int64_t)a.rows.B * a.pool.max_pages * 4);
        prefetch(a.q, line, (int64_t)a.rows.B * a.rows.n * a.rows.Hq * D * 2);
    }
    Walk at;
    int self = 0;
    if constexpr (ALONE) {
        at.b = blockIdx.x / (unsigned)sh.per_batch;
        at.i = blockIdx.x - at.b * sh.per_batch;
        at.nb = Line<Kv8AttnArgs>::blocks<false>(a, at.b);
        const int stagesful = (at.nb + NB - 1) / NB;
        at.t0 = stagesful * warp / W * NB;
        at.t1 = min(stagesful * (warp + 1) / W * NB, at.nb);
        at.left = at.t1 - at.t0;
        __syncthreads();                      // sm.abort is set
    } else {
        self = blockIdx.x * W + warp;
        if (!start_of_stretch(a, sh, warps, self, at)) return;   // behind it sm.abort is set
    }
    RawRows<D, NT> raw;
    bool first = true;
    fetch_rows<D, NT>(a, sh, decode_item(sh, a.pool.Hkv, at.b, at.i), raw);
    Walk &ahead = sm.ahead[warp];           // the same in every lane
    __syncwarp();
    ahead = at;
    __syncwarp();
    const WaitCtl wc{a.pool.err, &sm.abort, a.limit_ns};
    const int ps = a.pool.page_shift;
    // with one row tile a block is read once and makes way in L2 for what the join will read
    const uint64_t policy = sh.tiles == 1 ? tc::policy_evict_first() : policy_evict_normal();
    // The issuing side: each lane works out one of the next 32 blocks of a piece.
    int batch = 0, batch_n = 0;             // blocks of the batch issued, blocks in it (an even number)
    int next_t = ahead.t0;                  // next block of the piece to be worked out
    int src_row = 0, src_plane = 0;
    Meta src{NO_SLOT, 1.f, 1.f};
    unsigned issued = 0, taken = 0;         // stages
    int put = 0, get = 0, phase = 0;        // the ring's ends
    bool dead = false;
    auto refill = [&]() {                   // false: the stretch has no more blocks
        Walk w = ahead;
        while (w.valid() && next_t >= w.t1) {
            w.next(a, sh.per_batch);
            next_t = w.t0;
        }
        __syncwarp();
        ahead = w;
        __syncwarp();
        if (!w.valid()) return false;
        const int t = next_t + lane;
        src = Meta{NO_SLOT, 1.f, 1.f};
        if (t < w.t1) {
            const Item it = decode_item(sh, a.pool.Hkv, w.b, w.i);
            const int len = kv4_len(a.pool, w.b);
            const int64_t slot = (int64_t)Kv8Span(a, len).block(t) * KV8_BLOCK;
            if (slot < len) {
                const int id = kv4_page(a.pool, it.b, slot >> ps);
                if (id >= 0) {
                    src_row = (int)(slot & ((1 << ps) - 1));
                    src_plane = (int)kv8_plane(a.pool, id, it.h, 0);
                    src = Meta{(int)slot, *kv8_scale(a.pool, id, it.h, 0, src_row), *kv8_scale(a.pool, id, it.h, 1, src_row)};
                    // A block that no row sees (under vis) may never have been written.  Its weights
                    // are 0, but 0 times the 2^-e of such a scale could be NaN; its K scale only
                    // meets scores that the mask replaces.
                    if (!(src.v >= MIN_SCALE && src.v <= MAX_SCALE)) src.v = 1.f;
                }
            }
        }
        const int n = w.t1 - next_t;
        batch_n = n < 32 ? (n + NB - 1) / NB * NB : 32;
        batch = 0;
        next_t += 32;
        return true;
    };
    auto issue = [&]() {
        if (dead || (batch == batch_n && !refill())) return;
        if (lane >= batch && lane < batch + NB) {
            const uint32_t bar = smem_u32(&sm.full[warp][put]);
            sm.meta[warp][put][lane - batch] = src;
            if (src.slot != NO_SLOT) {
                const uint32_t dst = smem_u32(sm.ring[warp][put][lane - batch]);
                mbar_arrive_expect_tx(bar, 32 * D);
                tile_load(dst, &map, bar, src_row, src_plane, policy);
                tile_load(dst + 16 * D, &map, bar, src_row, src_plane + 1, policy);
            } else {
                mbar_arrive(bar);
            }
        }
        batch += NB;
        ++issued;
        if (++put == STAGES) put = 0;
    };
    for (int s = 0; s < STAGES; ++s) issue();
    __syncwarp();
    // a bound this short is the test hook's; the waits below can be met before it
    if (a.limit_ns < SHORT_WAIT_NS) dead = !waitw(smem_u32(&sm.hold), 0, wc);
    auto take = [&](const Item &it, const Rows<D, NT> &r, State<D, NT> &s, int blocks) {   // the next blocks of the ring
        float *scores = nullptr;
        const int srows = (int)score_rows(sh.rows);
        if (a.mass) scores = a.scores + ((((int64_t)it.b * a.pool.Hkv + it.h) * a.pool.max_pages) << ps) * srows;
        for (int t = 0; t < blocks; t += NB) {
            if (!dead && !waitw(smem_u32(&sm.full[warp][get]), phase, wc)) dead = true;
            if (dead) break;
            Meta mt[NB];
            bool any = false;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                mt[i] = sm.meta[warp][get][i];
                any |= mt[i].slot < r.max_limit;
            }
            if (any) blocks_step<D, NT>(sm.ring[warp][get][0], mt, r, a.sinks, scores, srows, it.tile * NT * 8, s);
            ++taken;
            if (++get == STAGES) get = 0, phase ^= 1;
            __syncwarp();                    // every lane has read the stage
            issue();
            __syncwarp();                    // ... and the slots are written before the next round reads them
        }
    };
    // after a wait that ran out: copies that were issued land before the block ends
    auto drain = [&] {
        const WaitCtl last{a.pool.err, &sm.never, a.drain_ns};
        for (; taken < issued; ++taken) {
            waitw(smem_u32(&sm.full[warp][get]), phase, last);
            if (++get == STAGES) get = 0, phase ^= 1;
        }
    };
    // the four elements d = D / 8 g + 4 j + {0..3} of column e of tile u
    auto four = [&](const State<D, NT> &s, int u, int j, int e) {
        return make_float4(s.o[u][2 * j][e], s.o[u][2 * j][e + 2], s.o[u][2 * j + 1][e], s.o[u][2 * j + 1][e + 2]);
    };
    if constexpr (ALONE) {
        Joined<D, NT, W> &jn = *reinterpret_cast<Joined<D, NT, W> *>(dyn + (sizeof(Smem<D, W>) + 15) / 16 * 16);
        const Item it = decode_item(sh, a.pool.Hkv, at.b, at.i);
        Rows<D, NT> r;
        make_rows<D, NT>(a, sh, it, kv4_len(a.pool, at.b), raw, r);
        State<D, NT> s;
        s.clear();
        take(it, r, s, at.t1 - at.t0);
        drain();
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = s.l[u][e];
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const int row = u * 8 + 2 * c + e;
                if (g == 0) jn.m[warp][row] = s.m[u][e], jn.l[warp][row] = l;
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    *reinterpret_cast<float4 *>(&jn.o[warp][row][D / 8 * g + 4 * j]) = four(s, u, j, e);
            }
        __syncthreads();
        for (int x = threadIdx.x; x < NT * 8 * (D / 4); x += W * 32) {
            const int row = x / (D / 4), d4 = x % (D / 4), rr = it.tile * NT * 8 + row;
            if (rr >= sh.rows) continue;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) m = fmaxf(m, jn.m[w][row]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = jn.m[w][row] == m ? 1.f : ex2(jn.m[w][row] - m);
                l = fmaf(f, jn.l[w][row], l);
                const float4 v = *reinterpret_cast<const float4 *>(&jn.o[w][row][d4 * 4]);
                o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
            }
            const int j = rr / sh.group, head = it.h * sh.group + rr % sh.group;
            const bool empty = l == 0.f;
            const float inv = empty ? 0.f : 1.f / l;
            put_out(a, (((int64_t)it.b * a.rows.n + j) * a.rows.Hq + head) * D + d4 * 4,
                    make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
            if (d4 == 0) a.lse[((int64_t)it.b * a.rows.Hq + head) * a.rows.n + j] = empty ? -INFINITY : fmaf(m, LN2, logf(l));
        }
        return;
    }
    for (; at.valid(); at.next(a, sh.per_batch)) {
        if (at.t0 >= at.t1) {                // the padding of an item that another warp has done
            first = false;
            continue;
        }
        const Item it = decode_item(sh, a.pool.Hkv, at.b, at.i);
        Rows<D, NT> r;
        if (!first) fetch_rows<D, NT>(a, sh, it, raw);
        first = false;
        make_rows<D, NT>(a, sh, it, kv4_len(a.pool, at.b), raw, r);
        State<D, NT> s;
        s.clear();
        take(it, r, s, at.t1 - at.t0);
        const bool whole = at.t0 == 0 && at.t1 == at.nb;
        float *part = static_cast<float *>(a.ws) + (2 * (int64_t)self + (at.t0 == 0 ? 1 : 0)) * Part<D, NT>::FLOATS;
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = s.l[u][e];
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const int row = u * 8 + 2 * c + e, rr = it.tile * NT * 8 + row;
                if (rr >= sh.rows) continue;
                const float m = s.m[u][e];
                if (!whole) {
                    if (g == 0) part[row] = m, part[8 * NT + row] = l;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        *reinterpret_cast<float4 *>(part + 16 * NT + row * D + D / 8 * g + 4 * j) = four(s, u, j, e);
                    continue;
                }
                const int j = rr / sh.group, head = it.h * sh.group + rr % sh.group;
                const bool empty = l == 0.f;
                const float inv = empty ? 0.f : 1.f / l;
                const int64_t at_out = (((int64_t)it.b * a.rows.n + j) * a.rows.Hq + head) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const float4 v = four(s, u, i, e);
                    put_out(a, at_out + D / 8 * g + 4 * i, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                }
                if (g == 0) a.lse[((int64_t)it.b * a.rows.Hq + head) * a.rows.n + j] = empty ? -INFINITY : fmaf(m, LN2, logf(l));
            }
    }
    drain();
}

// mass += the weights, from the scores that the attention kernel left (in L2, as far as they
// fit): a thread takes MASS_SLOTS slots with all their loads in flight (one slot at a time, in
// blocks of 256, took 8 x 16384 slots and 8 kv heads 2 us longer) and adds up the rows of its
// kv head in order.
constexpr int MASS_SLOTS = 4, MASS_CHUNK = MASS_SLOTS * 256;
constexpr int MASS_ROWS = 64;      // rows whose lse and range lie in shared memory at a time
__global__ void __launch_bounds__(256) kv8_mass_kernel(Kv8AttnArgs a, Shape sh, int chunks)
{
    __shared__ __align__(16) float lse2[MASS_ROWS];
    __shared__ int limit[MASS_ROWS], low[MASS_ROWS];
    const int chunk = (int)(blockIdx.x % (unsigned)chunks);
    const unsigned bh = blockIdx.x / (unsigned)chunks;
    const int b = (int)(bh / (unsigned)a.pool.Hkv), h = (int)(bh % (unsigned)a.pool.Hkv);
    const int srows = (int)score_rows(sh.rows);
    kv4_wait();
    kv4_trigger();   // as the join
    const int len = kv4_len(a.pool, b);
    const int64_t cap = (int64_t)a.pool.max_pages << a.pool.page_shift;
    for (int64_t s0 = (int64_t)chunk * MASS_CHUNK; s0 < len; s0 += (int64_t)chunks * MASS_CHUNK) {
        float *mass = a.mass + (int64_t)bh * cap + s0 + threadIdx.x;
        const float *x = a.scores + ((int64_t)bh * cap + s0 + threadIdx.x) * srows;
        float old[MASS_SLOTS], sum[MASS_SLOTS];
        int page[MASS_SLOTS];
        bool any[MASS_SLOTS];
#pragma unroll
        for (int i = 0; i < MASS_SLOTS; ++i) {
            const int64_t slot = s0 + threadIdx.x + 256 * i;
            old[i] = slot < len ? mass[256 * i] : 0.f;
            page[i] = slot < len ? a.pool.pages[(int64_t)b * a.pool.max_pages + (slot >> a.pool.page_shift)] : -1;
            sum[i] = 0.f;
            any[i] = false;
        }
        for (int r0 = 0; r0 < sh.rows; r0 += MASS_ROWS) {
            const int n = min(MASS_ROWS, sh.rows - r0);
            __syncthreads();
            bool whole = true;                               // the thread's row sees all slots in hand
            if ((int)threadIdx.x < n) {
                const int rr = r0 + threadIdx.x, j = rr / sh.group, head = h * sh.group + rr % sh.group;
                const int lim = kv4_limit(a.rows, b, j, len);
                limit[threadIdx.x] = lim;
                low[threadIdx.x] = a.window > 0 ? max(lim - a.window, 0) : 0;
                const float z = a.lse[((int64_t)b * a.rows.Hq + head) * a.rows.n + j];
                // a row of nothing but scores of -infinity gives no weight, and not NaN
                lse2[threadIdx.x] = z == -INFINITY ? INFINITY : z * LOG2E;
                whole = lim >= s0 + MASS_CHUNK && low[threadIdx.x] <= s0;
            } else if ((int)threadIdx.x < MASS_ROWS) {
                lse2[threadIdx.x] = INFINITY;                // rows that only fill up a four: weight 0
            }
            if (__syncthreads_and(whole)) {                  // most chunks
                for (int r = 0; r < n; r += 4) {
                    const float4 z = *reinterpret_cast<const float4 *>(lse2 + r);
                    float4 v[MASS_SLOTS];
#pragma unroll
                    for (int i = 0; i < MASS_SLOTS; ++i) v[i] = *reinterpret_cast<const float4 *>(x + (int64_t)256 * i * srows + r0 + r);
#pragma unroll
                    for (int i = 0; i < MASS_SLOTS; ++i) {   // row by row, as below
                        sum[i] += ex2(v[i].x - z.x);
                        sum[i] += ex2(v[i].y - z.y);
                        sum[i] += ex2(v[i].z - z.z);
                        sum[i] += ex2(v[i].w - z.w);
                        any[i] = true;
                    }
                }
                continue;
            }
            for (int r = 0; r < n; r += 4) {
                float4 v[MASS_SLOTS];
#pragma unroll
                for (int i = 0; i < MASS_SLOTS; ++i)
                    v[i] = s0 + threadIdx.x + 256 * i < len ? *reinterpret_cast<const float4 *>(x + (int64_t)256 * i * srows + r0 + r)
                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < MASS_SLOTS; ++i) {
                    const int64_t slot = s0 + threadIdx.x + 256 * i;
                    const float w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (r + e < n && slot < limit[r + e] && (slot >= low[r + e] || slot < a.sinks)) {
                            sum[i] += ex2(w[e] - lse2[r + e]);
                            any[i] = true;
                        }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MASS_SLOTS; ++i)
            if (any[i] && page[i] >= 0 && page[i] < a.pool.n_pages)   // slots of other pages have no scores
                mass[256 * i] = old[i] + sum[i];
    }
}

// Short tables: a block per item where the items fit the SMs at once, or twice over where they are of
// 512 tokens at most (8 kv heads, D = 128: 64 x 256 tokens 13.9 us where stretches and join take
// 17.5, 48 x 512 17.8 against 19.8, 64 ragged ones up to 512 14.0 against 13.3; 48 x 1024 27.9
// against 26.1, 64 ragged ones up to 1024 23.1 against 19.8, and 128 x 256, four times over, 25.2
// against 23.5).  The limits are the 4-bit kernel's.  Measured here, block per item against stretches
// and join (8 kv heads, 4 query heads each; D = 128 with one token, D = 64 with one, D = 64 with three,
// which is two tiles):
//   1 x 512     7.5 / 8.1     6.5 / 7.6     7.9 / 8.8       8 warps, up to 48 blocks
//   1 x 1024    10.1 / 8.3    8.4 / 7.7     10.5 / 9.1      8 warps, beyond
//   16 x 2048   16.7 / 20.9   12.7 / 15.7   16.3 / 20.5     8 warps, up to 128 blocks
//   24 x 1024   15.3 / 18.9   12.4 / 15.3   15.4 / 20.3     4 warps, up to 64 blocks
//   48 x 512    18.6 / 20.2   10.6 / 17.8   12.0 / 21.6     4 warps, up to 32 blocks (twice over with D = 128)
//   64 x 1024   30.0 / 31.5   16.7 / 21.0   30.5 / 30.7     4 warps (stretches, but with D = 64 and one token)
// and where the rule stays with stretches although a block per item is faster: 152 items of 3000 tokens
// 22.9 / 27.7, 256 items under a window of 1000 with 4 sinks (65 blocks) 16.5 / 22.4, ragged or not.
constexpr int ALONE_WARPS = 8, ALONE_BLOCKS = 48, ALONE_BLOCKS_MANY = 128, ALONE_BLOCKS_FULL = 64, ALONE_BLOCKS_TWICE = 32;

// The pool as [plane][row][D bytes], boxes of 16 rows.
bool make_pool_map(CUtensorMap *m, const Kv8Pool &pool, int D, int64_t n_pages)
{
    tc::EncodeFn enc = tc::get_encode();
    if (!enc) return false;
    const cuuint64_t page = 1ull << pool.page_shift;
    cuuint64_t dims[3] = {(cuuint64_t)D, page, (cuuint64_t)n_pages * pool.Hkv * 2};
    cuuint64_t strides[2] = {(cuuint64_t)D, page * D};
    cuuint32_t box[3] = {(cuuint32_t)D, 16, 1}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool.data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT>
int launch(const Kv8AttnArgs &a, const Shape &sh, const CUtensorMap &map, cudaStream_t st)
{
    constexpr int smem = sizeof(Smem<D, WARPS>);
    constexpr int alone = (sizeof(Smem<D, ALONE_WARPS>) + 15) / 16 * 16 + sizeof(Joined<D, NT, ALONE_WARPS>);
    constexpr int alone4 = (sizeof(Smem<D, WARPS>) + 15) / 16 * 16 + sizeof(Joined<D, NT, WARPS>);
    static_assert(alone <= 232448, "shared memory");
    // one block of the join per output row
    const int64_t joins = (int64_t)a.rows.B * (sh.per_batch / sh.tiles) * sh.rows;
    if (joins > 0x7fffffffLL) return CP_EUNSUPPORTED;
    // blocks of a grid that just fills the device, worked out once per device
    constexpr int MAX_DEV = 64;
    static std::atomic<int> fills[MAX_DEV], fills4[MAX_DEV];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEV) return CP_ECUDA;
    int fill = fills[dev].load(std::memory_order_acquire);
    if (!fill) {
        int resident = 0, resident4 = 0;
        const cudaFuncAttribute what = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if (cudaFuncSetAttribute(kv8_attn_kernel<D, NT, WARPS, false>, what, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kv8_attn_kernel<D, NT, WARPS, false>, WARPS * 32, smem) !=
                cudaSuccess ||
            resident < 1 ||
            cudaFuncSetAttribute(kv8_attn_kernel<D, NT, ALONE_WARPS, true>, what, alone) != cudaSuccess ||
            cudaFuncSetAttribute(kv8_attn_kernel<D, NT, WARPS, true>, what, alone4) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident4, kv8_attn_kernel<D, NT, WARPS, true>, WARPS * 32, alone4) !=
                cudaSuccess)
            return CP_ECUDA;
        fill = resident * sm_count();
        fills4[dev].store(resident4 * sm_count(), std::memory_order_relaxed);
        fills[dev].store(fill, std::memory_order_release);
    }
    const int64_t ctas = min(fill, part_rows(D) / (NT * 8 * WARPS));
    // an upper bound of an item's blocks from the sizes alone
    int64_t most = min((int64_t)a.pool.max_pages << (a.pool.page_shift - 4), (int64_t)1 << 27);
    if (a.window > 0 && !a.rows.vis)   // the sinks', the window's and the drafted tokens', each cut at both ends
        most = min(most, ((int64_t)a.sinks + 15) / 16 + ((int64_t)a.window + a.rows.n + 14) / 16 + 1);
    const int64_t items = (int64_t)a.rows.B * sh.per_batch, full = fills4[dev].load(std::memory_order_relaxed);
    cudaError_t rc;
    if (items <= sm_count() && most <= (2 * items >= sm_count() ? ALONE_BLOCKS_MANY : ALONE_BLOCKS)) {
        rc = kv4_launch(kv8_attn_kernel<D, NT, ALONE_WARPS, true>, (unsigned)items, ALONE_WARPS * 32, alone, st, map, a, sh, 0);
    } else if (items > sm_count() && ((items <= full && most <= ALONE_BLOCKS_FULL) || (items <= 2 * full && most <= ALONE_BLOCKS_TWICE))) {
        rc = kv4_launch(kv8_attn_kernel<D, NT, WARPS, true>, (unsigned)items, WARPS * 32, alone4, st, map, a, sh, 0);
    } else {
        const int64_t line = ((most > 0 ? most : 1) + PAD) * items;
        const int grid = (int)min(ctas, (line + LEAST * WARPS - 1) / (LEAST * WARPS));
        const int warps = grid * WARPS;
        if (kv4_launch(kv8_attn_kernel<D, NT, WARPS, false>, (unsigned)grid, WARPS * 32, smem, st, map, a, sh, warps) != cudaSuccess)
            return CP_ECUDA;
        // many warps where a row is cut into many pieces
        const int64_t cuts = warps / ((int64_t)a.rows.B * sh.per_batch);   // pieces of an item, about
        const unsigned n = (unsigned)joins;
        rc = cuts > 64   ? kv4_launch(kv_join_kernel<Kv8AttnArgs, D, NT, 16, 4>, n, 512, 0, st, a, sh, warps)
             : cuts > 16 ? kv4_launch(kv_join_kernel<Kv8AttnArgs, D, NT, 8, 8>, n, 256, 0, st, a, sh, warps)
             : cuts > 4  ? kv4_launch(kv_join_kernel<Kv8AttnArgs, D, NT, 4, 4>, n, 128, 0, st, a, sh, warps)
                         : kv4_launch(kv_join_rows_kernel<Kv8AttnArgs, D, NT, 4>, (n + 3) / 4, 128, 0, st, a, sh, warps, (int)n);
    }
    if (rc != cudaSuccess) return CP_ECUDA;
    if (!a.mass) return CP_OK;
    // enough blocks to fill the device a few times; longer tables are walked
    const int64_t heads = (int64_t)a.rows.B * a.pool.Hkv, cap = (int64_t)a.pool.max_pages << a.pool.page_shift;
    int64_t chunks = (cap + MASS_CHUNK - 1) / MASS_CHUNK;
    const int64_t enough = ((int64_t)sm_count() * 32 + heads - 1) / heads;
    if (chunks > enough) chunks = enough;
    if (chunks < 1) return CP_OK;
    if (heads * chunks > 0x7fffffffLL) return CP_EUNSUPPORTED;
    return kv4_launch(kv8_mass_kernel, (unsigned)(heads * chunks), 256, 0, st, a, sh, (int)chunks) == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace

// The warps' parts, then the scores.
size_t kv8_attn_workspace_bytes(int B, int n, int Hq, int Hkv, int D, int64_t slots, bool mass)
{
    if (D != 64 && D != 128) return 0;
    const size_t parts = (size_t)2 * part_rows(D) * (D + 2) * sizeof(float);
    if (!mass) return parts;
    const int64_t rows = score_rows((int64_t)n * (Hq / Hkv));
    const unsigned __int128 b = (unsigned __int128)(unsigned)B * (unsigned)Hkv * (uint64_t)rows * (uint64_t)slots * 4u;
    if (b > ((unsigned __int128)1 << 61)) return 0;
    return parts + (((size_t)b + 255) & ~(size_t)255);
}

int launch_kv8_attn(const Kv8AttnArgs &given, int D, int64_t n_pages, cudaStream_t st)
{
    Kv8AttnArgs a = given;
    if (a.mass) a.scores = static_cast<float *>(a.ws) + (size_t)2 * part_rows(D) * (D + 2);
    Shape sh;
    sh.group = a.rows.Hq / a.pool.Hkv;
    const int64_t rows = (int64_t)a.rows.n * sh.group;
    const int nt = rows > 8 ? 2 : 1;
    const int64_t tiles = (rows + nt * 8 - 1) / (nt * 8);
    const int64_t per = tiles * a.pool.Hkv;
    if (rows > 0x3fffffffLL || per > 0x3fffffffLL) return CP_EUNSUPPORTED;
    if (n_pages * a.pool.Hkv * 2 > 0x7fffffffLL) return CP_EUNSUPPORTED;
    sh.rows = (int)rows;
    sh.tiles = (int)tiles;
    sh.per_batch = (int)per;
    CUtensorMap map{};
    if (n_pages > 0 && !make_pool_map(&map, a.pool, D, n_pages)) return CP_ECUDA;
    if (D == 64) return nt == 1 ? launch<64, 1>(a, sh, map, st) : launch<64, 2>(a, sh, map, st);
    return nt == 1 ? launch<128, 1>(a, sh, map, st) : launch<128, 2>(a, sh, map, st);
}

}  // namespace cp
