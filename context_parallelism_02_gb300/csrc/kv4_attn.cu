// kv4_attn.cu -- attention of a few query tokens over the paged 4-bit cache.
//
//   s_ij = scale q_i . k_j over the slots j that row i sees,
//   lse_i = ln sum_j e^{s_ij},   out_i = sum_j e^{s_ij - lse_i} v_j;
//   a row that sees nothing: (0, -inf).
//
// HBM-bound for few query rows: a token and kv head is 1.25 D bytes, read once
// for all rows of the tile.  The work of a 16-token block is two products on
// mma.m16n8k16 with the cache as the A operand, S^T = K q^T and O^T += V^T P^T:
// 16 tokens (or 16 d) by 8 query rows, so that the few rows of a decode step fill
// the narrow side of the instruction, and a lane unpacks exactly the codes it
// feeds to the tensor core, in registers.
//
// Scores: with n the code, s_ij = sum_gr [ s_jgr sum_d n q_d + m_jgr sum_d q_d ].
// A masked nibble is an fp16 as it stands: a subnormal, n 2^-24 in the lowest four
// bits and 16 n 2^-24 in the next four (their elements of q are divided by 16), so
// unpacking K is one AND a pair.  q is scaled per row by a power of two into fp16's
// range: its largest element comes to 2^8 (2^4 where it is divided by 16), bf16's 8 bits
// fit down to 2^-21 of it, and the products are exact; smaller elements are off by up to
// 2^-29 of the largest.  The group's scale multiplies an fp32 sum.  The minima are one
// more product, m (fp16, exact) with the rows' group sums of q in three fp16 parts.
// V's values s n + m are rounded to fp16 (relative 2^-11, below 2^-14 absolute 2^-25)
// and so are the weights P; the row sums are taken over the unrounded fp32 weights.
// Weights are relative to a reference 7 to 15 powers of two below the largest score of the
// stretch so far, so that the largest weight is 2^7 to 2^15 and a small one is off by 2^-11
// of itself or 2^-32 of the largest: a long tail behind one large score is not lost from
// O while it counts in the sums.  V and P in one fp16 part each are a choice: a second
// part of either doubles the 8 products of a block in a kernel that is short of issue slots,
// and what it would mend is below the output's own bf16 step (error against 64 bits 0.0017
// of the outputs' norm either way; one output in 8 falls on the other side of a bf16 step).
//
// Measured (Hq = 32, Hkv = 8, D = 128): 16 x 32768 tokens 119.5 us, 5.6 TB/s of cache,
// 108 without the arithmetic; 4 x 32768 37.6 us; 1 x 512 (a block per item) 7.0 us.  Per block 340
// instructions: the integer pipe and the heavy half of the FMA pipe take 60 cycles of
// an SM each, issue 85, HBM at its copy rate 112.
#include <atomic>

#include "kernels.h"
#include "kv4.cuh"
#include "kv_line.cuh"
#include "tc_helpers.cuh"

// Schedule.  All items' blocks of 16 tokens form one line, batch by batch and
// item by item, and every warp of a grid that just fills the GPU takes an equal
// stretch of it, whatever the lengths: lengths are read on the device, so a
// captured step stays balanced as the sequences grow.  An item counts PAD blocks
// more than it has, for what a warp spends on starting and ending it.  A stretch
// is cut into pieces at the items' ends; a piece that is a whole item is written
// out, the others leave partial sums that a second kernel joins by log-sum-exp, in
// the order of the line (no atomics: results repeat bit for bit).  Warps share
// nothing: each has its own ring of shared-memory stages filled by bulk copies.
// Short tables of few items take a block per item instead (ALONE).
namespace cp {

template <>
struct Line<Kv4AttnArgs> {
    // with 4, 64 ragged sequences up to 8192 tokens take 38 us instead of 33, with 16 34
    static constexpr int PAD = 8;
    static constexpr int LEAST = 2;   // a stage (512 tokens: 8.5 us, with 4 9.0)
    static constexpr bool NEXT_EARLY = true;
    template <bool EARLY>
    __device__ __forceinline__ static int blocks(const Kv4AttnArgs &a, int b)
    {
        if (a.sel) return a.n_sel << (a.pool.page_shift - 4);
        const int len = kv4_len<EARLY>(a.pool, b);
        return len > 0 ? (len - 1) / KV4_BLOCK + 1 : 1;
    }
};

namespace {

constexpr int WARPS = 4;
constexpr int PAD = Line<Kv4AttnArgs>::PAD, LEAST = Line<Kv4AttnArgs>::LEAST;

__device__ __forceinline__ int item_blocks(const Kv4AttnArgs &a, int b) { return Line<Kv4AttnArgs>::blocks<false>(a, b); }


// (w & mask) | magic in one instruction (as immediates the compiler makes two of it,
// and the integer pipe bounded the kernel: 16 x 32768 tokens 150 us, 130 with this).
__device__ __forceinline__ __half2 pick(uint32_t w, uint32_t mask)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
    return as_h2(r);
}

// The four code pairs of a word (nibbles e, e + 4 of the low and high half) as the
// subnormal fp16 pairs n 2^-24, 16 n 2^-24, n 2^-24, 16 n 2^-24.
__device__ __forceinline__ void unpack_raw(uint32_t w, uint32_t (&n)[4])
{
    const uint32_t u = w >> 8;
    n[0] = w & 0x000f000fu;
    n[1] = w & 0x00f000f0u;
    n[2] = u & 0x000f000fu;
    n[3] = u & 0x00f000f0u;
}

// The same as exact fp16 pairs n: a nibble in the low bits of an fp16 of exponent 2^10 reads
// 1024 + n, in the next four bits 1024 + 16 n.
__device__ __forceinline__ void unpack(uint32_t w, __half2 (&n)[4])
{
    const __half2 k1024 = __float2half2_rn(1024.f), k16 = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.f);
    const uint32_t u = w >> 8;
    n[0] = __hsub2(pick(w, 0x000f000fu), k1024);
    n[1] = __hfma2(pick(w, 0x00f000f0u), k16, k64);
    n[2] = __hsub2(pick(u, 0x000f000fu), k1024);
    n[3] = __hfma2(pick(u, 0x00f000f0u), k16, k64);
}

// Query rows of one tile, as B operands, and what goes with a row.  Lane (g, c) =
// (lane / 4, lane % 4) holds row 8 t + g's share in q; the accumulators' columns
// are rows 8 t + 2c and 8 t + 2c + 1.
template <int D, int NT>
struct Rows {
    static constexpr int NG = Kv4<D>::NG;
    uint32_t q[NT][NG][4];     // group gr: elements 8 c + {0,1}, {2,3} / 16, {4,5}, {6,7} / 16
    uint32_t sum[NT][2];       // group c: hi, mid | lo, 0 of the sum of q
    float to_log2[NT][2];      // score -> log2 units, for the lane's two columns
    int limit[NT][2];          // slots that the column's row sees
    int min_limit, max_limit;  // over the tile
};

// Running state of a warp: m in log2 units (a lazily raised reference, 7 to 15 below the
// maximum), l per lane (its own tokens), O^T accumulators.
template <int D, int NT>
struct State {
    static constexpr int NG = Kv4<D>::NG;
    float m[NT][2], l[NT][2];
    float o[NT][2 * NG][4];    // tile 2 gr + (e >> 1), element (e & 1) 2 + column: d = 32 gr + 4 g + e
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
        }
    }
};

// A lane's share of the rows as they are in memory, so that their latency can
// overlap with other loads.
template <int D, int NT>
struct RawRows {
    uint4 w[NT][Kv4<D>::NG];
};

template <int D, int NT>
__device__ __forceinline__ void fetch_rows(const Kv4AttnArgs &a, const Shape &sh, const Item &it, RawRows<D, NT> &raw)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = (it.tile * NT + t) * 8 + g;
        const bool on = row < sh.rows;
        const int j = it.j0 + (on ? row / sh.group : 0);
        const int head = it.h * sh.group + (on ? row % sh.group : 0);
        const uint4 *p = reinterpret_cast<const uint4 *>(a.q + (((int64_t)it.b * a.rows.n + j) * a.rows.Hq + head) * D);
#pragma unroll
        for (int gr = 0; gr < Kv4<D>::NG; ++gr) raw.w[t][gr] = on ? p[gr * 4 + c] : make_uint4(0, 0, 0, 0);
    }
}

template <int D, int NT>
__device__ __forceinline__ void make_rows(const Kv4AttnArgs &a, const Shape &sh, const Item &it, int len,
                                          const RawRows<D, NT> &raw, Rows<D, NT> &r)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    int lo = 0x7fffffff, hi = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = (it.tile * NT + t) * 8 + g;
        const bool on = row < sh.rows;
        const int j = it.j0 + (on ? row / sh.group : 0);
        const uint4(&w)[NG] = raw.w[t];
        float top = 0.f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            const uint32_t x[4] = {w[gr].x, w[gr].y, w[gr].z, w[gr].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // q 2^sh has its largest magnitude in [2^8, 2^9): group sums stay below 2^14
        int sh2 = 0;
        if (top > 0.f && top < INFINITY) sh2 = 8 - ilogbf(top);
        sh2 = sh2 > 120 ? 120 : sh2;
        const float up = __int_as_float((127 + (sh2 < -126 ? -126 : sh2)) << 23);
        float sum = 0.f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            const uint32_t x[4] = {w[gr].x, w[gr].y, w[gr].z, w[gr].w};
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = i & 1 ? up * 0.0625f : up;
                const __half2 v = __floats2half2_rn(__uint_as_float(x[i] << 16) * f, __uint_as_float(x[i] & 0xffff0000u) * f);
                r.q[t][gr][i] = h2(v);
                const float both = __low2float(v) + __high2float(v);
                part += i & 1 ? both * 16.f : both;
            }
            part += __shfl_xor_sync(0xffffffffu, part, 1);
            part += __shfl_xor_sync(0xffffffffu, part, 2);
            if (gr == c) sum = part;
        }
        const __half s0 = __float2half_rn(sum);
        const float r1 = sum - __half2float(s0);
        const __half s1 = __float2half_rn(r1);
        const __half s2 = __float2half_rn(r1 - __half2float(s1));
        r.sum[t][0] = h2(__halves2half2(s0, s1));
        r.sum[t][1] = h2(__halves2half2(s2, __ushort_as_half(0)));
        const float back = a.scale * LOG2E * (16777216.f / up);   // scores are in units of 2^-24 up
        const int lim = on ? kv4_limit(a.rows, it.b, j, len) : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            r.to_log2[t][e] = __shfl_sync(0xffffffffu, back, (2 * c + e) * 4);
            r.limit[t][e] = __shfl_sync(0xffffffffu, lim, (2 * c + e) * 4);
        }
        lo = min(lo, on ? lim : 0x7fffffff);
        hi = max(hi, lim);
    }
    r.min_limit = __reduce_min_sync(0xffffffffu, lo);
    r.max_limit = __reduce_max_sync(0xffffffffu, hi);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N])
{
    static_assert(N == 2 || N == 4, "");
    if (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[N - 2] = v.z, w[N - 1] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

// Scores of one block, in units of the row's to_log2: x[t][0..1] token g, x[t][2..3] token g + 8.
template <int D, int NT>
__device__ __forceinline__ void block_scores(const uint8_t *blk, const Rows<D, NT> &r, float (&x)[NT][4])
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint32_t ka[NG], kb[NG], ma[NG], mb[NG];
    load_words<NG>(blk + g * (D / 2) + c * 4 * NG, ka);
    load_words<NG>(blk + (g + 8) * (D / 2) + c * 4 * NG, kb);
    load_words<NG>(blk + Kv4<D>::K_META + g * 4 * NG, ma);
    load_words<NG>(blk + Kv4<D>::K_META + (g + 8) * 4 * NG, mb);
    // the minima of group c as both halves of a pair (k = 2c, 2c+1 and 2c+8, 2c+9)
    uint32_t na = 0, nb = 0;
    if (NG == 4 || c < NG) {
        na = *reinterpret_cast<const uint16_t *>(blk + Kv4<D>::K_META + (g * NG + c) * 4 + 2) * 0x10001u;
        nb = *reinterpret_cast<const uint16_t *>(blk + Kv4<D>::K_META + ((g + 8) * NG + c) * 4 + 2) * 0x10001u;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        mma16816_zero(x[t], na, nb, na, nb, r.sum[t][0], r.sum[t][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] *= 1.f / 16777216.f;   // the codes' unit, 2^-24
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
        uint32_t u[4], v[4];
        unpack_raw(ka[gr], u);
        unpack_raw(kb[gr], v);
        const float sa = __low2float(as_h2(ma[gr])), sb = __low2float(as_h2(mb[gr]));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float acc[4];
            mma16816_zero(acc, u[0], v[0], u[1], v[1], r.q[t][gr][0], r.q[t][gr][1]);
            mma16816(acc, u[2], v[2], u[3], v[3], r.q[t][gr][2], r.q[t][gr][3]);
            x[t][0] = fmaf(sa, acc[0], x[t][0]);
            x[t][1] = fmaf(sa, acc[1], x[t][1]);
            x[t][2] = fmaf(sb, acc[2], x[t][2]);
            x[t][3] = fmaf(sb, acc[3], x[t][3]);
        }
    }
}

// The references m lie this far below the largest score when they are raised, and are
// raised where a score passes them by more than 15: 2^15 is an fp16.
constexpr float BELOW = 7.f, LAG = 15.f;

template <int D, int NT, int NB>
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
            for (int i = 0; i < 2 * Kv4<D>::NG; ++i) s.o[t][i][e] *= f, s.o[t][i][e + 2] *= f;
        }
}

// V^T fragments of group gr of a block: f[e][half], e = 0..3 the elements
// 32 gr + 4 g + e.
template <int D>
__device__ __forceinline__ void value_frags(const uint32_t (&w)[2], const uint2 (&sm)[2], uint32_t (&f)[4][2])
{
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        __half2 n[4];
        unpack(w[hf], n);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e][hf] = h2(__hfma2(n[e], as_h2(sm[hf].x), as_h2(sm[hf].y)));
    }
}

// O^T += V^T P^T for one block, p the weights as B operands.  CUT: some row does
// not see all of the block's tokens.  A token that no row sees (at or past `live`)
// may hold anything, and one that only some rows see may hold NaN, which 0 times
// would carry to the others: both count as 0, and the rows that do see a NaN get
// it afterwards.  rel: the rows' limits from the block's first slot.
template <int D, int NT, bool CUT>
__device__ __forceinline__ void block_values(const uint8_t *blk, int live, const int (&rel)[NT][2],
                                             const uint32_t (&p)[NT][2], State<D, NT> &s)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, c = lane & 3;
    uint32_t w[2][NG];
    uint2 sm[2][NG];
    uint32_t nan[NG];   // tokens whose group is NaN
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        load_words<NG>(blk + Kv4<D>::V_CODES + hf * 128 * NG + lane * 4 * NG, w[hf]);
#pragma unroll
        for (int gr = 0; gr < NG; gr += 2) {
            const uint4 v = *reinterpret_cast<const uint4 *>(blk + Kv4<D>::V_META + ((hf * 4 + c) * NG + gr) * 8);
            sm[hf][gr] = make_uint2(v.x, v.y);
            sm[hf][gr + 1] = make_uint2(v.z, v.w);
        }
        if (CUT) {
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                if (hf == 0) nan[gr] = 0;
                uint2 &v = sm[hf][gr];
#pragma unroll
                for (int lo = 0; lo < 2; ++lo) {
                    const int k = hf * 8 + 2 * c + lo;
                    const uint32_t half = lo ? 0xffff0000u : 0x0000ffffu, exps = half & 0x7c007c00u;
                    const bool bad = (v.x & exps) == exps || (v.y & exps) == exps;
                    if (bad || k >= live) v.x &= ~half, v.y &= ~half;
                    const unsigned who = __ballot_sync(0xffffffffu, bad && k < live);   // lanes c of every g alike
#pragma unroll
                    for (int i = 0; i < 4; ++i) nan[gr] |= (who >> i & 1u) << (hf * 8 + 2 * i + lo);
                }
            }
        }
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
        const uint32_t wg[2] = {w[0][gr], w[1][gr]};
        const uint2 mg[2] = {sm[0][gr], sm[1][gr]};
        uint32_t f[4][2];
        value_frags<D>(wg, mg, f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mma16816(s.o[t][2 * gr], f[0][0], f[1][0], f[0][1], f[1][1], p[t][0], p[t][1]);
            mma16816(s.o[t][2 * gr + 1], f[2][0], f[3][0], f[2][1], f[3][1], p[t][0], p[t][1]);
        }
        if (CUT && nan[gr]) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = rel[t][e] < 0 ? 0 : rel[t][e] > 16 ? 16 : rel[t][e];
                    if (nan[gr] & ((1u << n) - 1u)) s.o[t][2 * gr][e] = s.o[t][2 * gr][e + 2] = s.o[t][2 * gr + 1][e] =
                        s.o[t][2 * gr + 1][e + 2] = __int_as_float(0x7fffffff);
                }
        }
    }
}

// NB blocks of 16 tokens, block i beginning at slot[i], for the warp's state.
template <int D, int NT, int NB>
__device__ __forceinline__ void blocks_step(const uint8_t *blk, const int (&slot)[NB], const Rows<D, NT> &r, State<D, NT> &s)
{
    const int lane = threadIdx.x & 31, g = lane >> 2;
    float x[NB][NT][4];
    bool cut = false;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        block_scores<D, NT>(blk + i * Kv4<D>::BYTES, r, x[i]);
        cut |= slot[i] > r.min_limit - KV4_BLOCK;
        // rounded here and not fused with the subtraction of m, which is one of these
        // products: a difference is then at most LAG however large the scores are
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][t][e] = __fmul_rn(x[i][t][e], r.to_log2[t][e & 1]);
    }
    if (cut) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (slot[i] + g + (e >> 1) * 8 >= r.limit[t][e & 1]) x[i][t][e] = -INFINITY;
    }
    raise_max<D, NT, NB>(x, s);
    uint32_t p[NB][NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) base[e] = s.m[t][e] == -INFINITY ? 0.f : -s.m[t][e];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = ex2(__fadd_rn(x[i][t][e], base[e & 1]));
                s.l[t][e & 1] += w[e];
            }
            p[i][t][0] = movmatrix(h2(__floats2half2_rn(w[0], w[1])));
            p[i][t][1] = movmatrix(h2(__floats2half2_rn(w[2], w[3])));
        }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const uint8_t *b = blk + i * Kv4<D>::BYTES;
        const int live = r.max_limit - slot[i];
        int rel[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) rel[t][0] = r.limit[t][0] - slot[i], rel[t][1] = r.limit[t][1] - slot[i];
        if (!cut) block_values<D, NT, false>(b, live, rel, p[i], s);
        else if (live > 0) block_values<D, NT, true>(b, live, rel, p[i], s);
    }
}

constexpr int NB = 2;      // blocks of a stage, taken together

// Stages of a warp's ring.  12 warps an SM with one stage of 5 KB on the way and one in
// hand cover latency x bandwidth (46 KB an SM); more on the way is slower (16 x 32768
// tokens: 2 stages 117 us, 3 120, 4 130).
template <int D>
__host__ __device__ constexpr int stages() { return 2; }

template <int D, int W>
struct Smem {
    uint8_t ring[W][stages<D>()][NB][Kv4<D>::BYTES];
    uint64_t full[W][stages<D>()];
    uint64_t hold;                   // completed by nobody: what the failure path is tested with
    int slot[W][stages<D>()][NB];   // first slot of the block, or NO_SLOT
    Walk ahead[W];               // the piece that a warp's copies are issued for
    int abort, never;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// ALONE: a block per item, its W warps share the item's blocks evenly and join in
// shared memory, and there is no second kernel (short tables); else the schedule at the
// top of this file.
template <int D, int NT, int W, bool ALONE>
__global__ void __launch_bounds__(W * 32) kv4_attn_kernel(Kv4AttnArgs a, Shape sh, int warps)
{
    extern __shared__ __align__(128) uint8_t dyn[];
    Smem<D, W> &sm = *reinterpret_cast<Smem<D, W> *>(dyn);
    constexpr int NS = stages<D>(), NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    if (lane < NS) mbar_init(smem_u32(&sm.full[warp][lane]), NB);
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
        if (a.sel) prefetch(a.sel, line, (int64_t)a.rows.B * a.rows.n * a.pool.Hkv * a.n_sel * 4);
    }
    Walk at;
    int self = 0;
    if constexpr (ALONE) {
        at.b = blockIdx.x / (unsigned)sh.per_batch;
        at.i = blockIdx.x - at.b * sh.per_batch;
        at.nb = item_blocks(a, at.b);
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
    const int ps = a.pool.page_shift, bpp = 1 << (ps - 4);
    // with one row tile a block is read once and makes way in L2 for what the join
    // will read (4 x 32k tokens: 39.8 us without, 37.3 us with)
    const uint64_t policy = sh.tiles == 1 ? tc::policy_evict_first() : policy_evict_normal();
    // The issuing side: each lane works out one of the next 32 blocks of a piece.
    int batch = 0, batch_n = 0;             // blocks of the batch issued, blocks in it (an even number)
    int next_t = ahead.t0;                  // next block of the piece to be worked out
    const uint8_t *src = nullptr;
    int src_slot = NO_SLOT;
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
        src = nullptr;
        src_slot = NO_SLOT;
        if (t < w.t1) {
            const Item it = decode_item(sh, a.pool.Hkv, w.b, w.i);
            const int len = kv4_len(a.pool, w.b);
            int lp = t >> (ps - 4);
            bool on = true;
            if (a.sel) {
                lp = a.sel[(((int64_t)it.b * a.rows.n + it.j0) * a.pool.Hkv + it.h) * a.n_sel + lp];
                on = lp >= 0;
                if (on && lp > (len - 1) >> ps) {   // len 0: -1 >> ps is -1
                    kv4_report(a.pool.err);
                    on = false;
                }
            }
            const int64_t slot = ((int64_t)lp << ps) + (t & (bpp - 1)) * KV4_BLOCK;
            if (on && slot < len) {
                const int id = kv4_page(a.pool, it.b, lp);
                if (id >= 0) {
                    src = kv4_block<D>(a.pool, id, it.h, t & (bpp - 1));
                    src_slot = (int)slot;
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
            sm.slot[warp][put][lane - batch] = src_slot;
            if (src) {
                mbar_arrive_expect_tx(bar, Kv4<D>::BYTES);
                bulk_load(smem_u32(sm.ring[warp][put][lane - batch]), src, Kv4<D>::BYTES, bar, policy);
            } else {
                mbar_arrive(bar);
            }
        }
        batch += NB;
        ++issued;
        if (++put == NS) put = 0;
    };
    for (int s = 0; s < NS; ++s) issue();
    __syncwarp();
    // a bound this short is the test hook's; the waits below can be met before it
    if (a.limit_ns < SHORT_WAIT_NS) dead = !waitw(smem_u32(&sm.hold), 0, wc);
    auto take = [&](const Rows<D, NT> &r, State<D, NT> &s, int blocks) {   // the next blocks of the ring
        for (int t = 0; t < blocks; t += NB) {
            if (!dead && !waitw(smem_u32(&sm.full[warp][get]), phase, wc)) dead = true;
            if (dead) break;
            int slot[NB];
            bool any = false;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                slot[i] = sm.slot[warp][get][i];
                any |= slot[i] < r.max_limit;
            }
            if (any) blocks_step<D, NT, NB>(sm.ring[warp][get][0], slot, r, s);
            ++taken;
            if (++get == NS) get = 0, phase ^= 1;
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
            if (++get == NS) get = 0, phase ^= 1;
        }
    };
    if constexpr (ALONE) {
        Joined<D, NT, W> &jn = *reinterpret_cast<Joined<D, NT, W> *>(dyn + (sizeof(Smem<D, W>) + 15) / 16 * 16);
        const Item it = decode_item(sh, a.pool.Hkv, at.b, at.i);
        Rows<D, NT> r;
        make_rows<D, NT>(a, sh, it, kv4_len(a.pool, at.b), raw, r);
        State<D, NT> s;
        s.clear();
        take(r, s, at.t1 - at.t0);
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
                for (int gr = 0; gr < NG; ++gr)
                    *reinterpret_cast<float4 *>(&jn.o[warp][row][32 * gr + 4 * g]) = make_float4(
                        s.o[u][2 * gr][e], s.o[u][2 * gr][e + 2], s.o[u][2 * gr + 1][e], s.o[u][2 * gr + 1][e + 2]);
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
            const int j = it.j0 + rr / sh.group, head = it.h * sh.group + rr % sh.group;
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
        take(r, s, at.t1 - at.t0);
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
                    for (int gr = 0; gr < NG; ++gr)
                        *reinterpret_cast<float4 *>(part + 16 * NT + row * D + 32 * gr + 4 * g) = make_float4(
                            s.o[u][2 * gr][e], s.o[u][2 * gr][e + 2], s.o[u][2 * gr + 1][e], s.o[u][2 * gr + 1][e + 2]);
                    continue;
                }
                const int j = it.j0 + rr / sh.group, head = it.h * sh.group + rr % sh.group;
                const bool empty = l == 0.f;
                const float inv = empty ? 0.f : 1.f / l;
                const int64_t at_out = (((int64_t)it.b * a.rows.n + j) * a.rows.Hq + head) * D;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
                    put_out(a, at_out + 32 * gr + 4 * g, make_float4(s.o[u][2 * gr][e] * inv, s.o[u][2 * gr][e + 2] * inv,
                                                                     s.o[u][2 * gr + 1][e] * inv, s.o[u][2 * gr + 1][e + 2] * inv));
                if (g == 0) a.lse[((int64_t)it.b * a.rows.Hq + head) * a.rows.n + j] = empty ? -INFINITY : fmaf(m, LN2, logf(l));
            }
    }
    drain();
}

// Short tables: a block per item where the items fit the SMs at once.  8 items of 512
// tokens take 7.0 us (by stretches and join 8.4), of 1024 9.4 (8.5); 128 items of 512
// 7.3 us (14.0), of 1024 9.9 (15.3), of 2048 14.7 (18.5).  More items than SMs: blocks
// of four warps as long as they fit at once; 256 items of 512 tokens 11.3 us (15.6), of
// 1024 17.1 (19.9), of 2048 29.0 (25.1), 448 of 1024 18.3 (26.7).
constexpr int ALONE_WARPS = 8, ALONE_BLOCKS = 48, ALONE_BLOCKS_MANY = 128, ALONE_BLOCKS_FULL = 64;
template <int D, int NT>
int launch(const Kv4AttnArgs &a, const Shape &sh, cudaStream_t st)
{
    constexpr int smem = sizeof(Smem<D, WARPS>);
    constexpr int alone = (sizeof(Smem<D, ALONE_WARPS>) + 15) / 16 * 16 + sizeof(Joined<D, NT, ALONE_WARPS>);
    constexpr int alone4 = (sizeof(Smem<D, WARPS>) + 15) / 16 * 16 + sizeof(Joined<D, NT, WARPS>);
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
        if (cudaFuncSetAttribute(kv4_attn_kernel<D, NT, WARPS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kv4_attn_kernel<D, NT, WARPS, false>, WARPS * 32, smem) != cudaSuccess ||
            resident < 1 ||
            cudaFuncSetAttribute(kv4_attn_kernel<D, NT, ALONE_WARPS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, alone) !=
                cudaSuccess ||
            cudaFuncSetAttribute(kv4_attn_kernel<D, NT, WARPS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, alone4) !=
                cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident4, kv4_attn_kernel<D, NT, WARPS, true>, WARPS * 32, alone4) !=
                cudaSuccess)
            return CP_ECUDA;
        fill = resident * sm_count();
        fills4[dev].store(resident4 * sm_count(), std::memory_order_relaxed);
        fills[dev].store(fill, std::memory_order_release);
    }
    const int64_t ctas = min(fill, MAX_ROWS / (NT * 8 * WARPS));
    // an upper bound of the line from the sizes alone (a length is below 2^31: 2^27 blocks)
    const int64_t most = a.sel ? (int64_t)a.n_sel << (a.pool.page_shift - 4)
                               : min((int64_t)a.pool.max_pages << (a.pool.page_shift - 4), (int64_t)1 << 27);
    const int64_t items = (int64_t)a.rows.B * sh.per_batch;
    if (items <= sm_count() && most <= (2 * items >= sm_count() ? ALONE_BLOCKS_MANY : ALONE_BLOCKS)) {
        const cudaError_t rc = kv4_launch(kv4_attn_kernel<D, NT, ALONE_WARPS, true>, (unsigned)items,
                                          ALONE_WARPS * 32, alone, st, a, sh, 0);
        return rc == cudaSuccess ? CP_OK : CP_ECUDA;
    }
    if (items > sm_count() && items <= fills4[dev].load(std::memory_order_relaxed) && most <= ALONE_BLOCKS_FULL) {
        const cudaError_t rc =
            kv4_launch(kv4_attn_kernel<D, NT, WARPS, true>, (unsigned)items, WARPS * 32, alone4, st, a, sh, 0);
        return rc == cudaSuccess ? CP_OK : CP_ECUDA;
    }
    const int64_t line = ((most > 0 ? most : 1) + PAD) * items;
    const int grid = (int)min(ctas, (line + LEAST * WARPS - 1) / (LEAST * WARPS));
    const int warps = grid * WARPS;
    if (kv4_launch(kv4_attn_kernel<D, NT, WARPS, false>, (unsigned)grid, WARPS * 32, smem, st, a, sh, warps) != cudaSuccess)
        return CP_ECUDA;
    // many warps where a row is cut into many pieces
    const int64_t cuts = warps / ((int64_t)a.rows.B * sh.per_batch);   // pieces of an item, about
    const unsigned n = (unsigned)joins;
    const cudaError_t rc =
        cuts > 64  ? kv4_launch(kv_join_kernel<Kv4AttnArgs, D, NT, 16, 4>, n, 512, 0, st, a, sh, warps)
        : cuts > 16 ? kv4_launch(kv_join_kernel<Kv4AttnArgs, D, NT, 8, 8>, n, 256, 0, st, a, sh, warps)
                    : kv4_launch(kv_join_kernel<Kv4AttnArgs, D, NT, 4, 4>, n, 128, 0, st, a, sh, warps);
    return rc == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace

size_t kv4_attn_workspace_bytes(int D)
{
    if (D != 64 && D != 128) return 0;
    return (size_t)2 * MAX_ROWS * (D + 2) * sizeof(float);
}

int launch_kv4_attn(const Kv4AttnArgs &a, int D, cudaStream_t st)
{
    Shape sh;
    sh.group = a.rows.Hq / a.pool.Hkv;
    const int64_t rows = (int64_t)(a.sel ? 1 : a.rows.n) * sh.group;
    const int nt = rows > 8 ? 2 : 1;
    const int64_t tiles = (rows + nt * 8 - 1) / (nt * 8);
    const int64_t per = (a.sel ? a.rows.n : 1) * tiles * a.pool.Hkv;
    if (rows > 0x3fffffffLL || per > 0x3fffffffLL) return CP_EUNSUPPORTED;
    sh.rows = (int)rows;
    sh.tiles = (int)tiles;
    sh.per_batch = (int)per;
    if (D == 64) return nt == 1 ? launch<64, 1>(a, sh, st) : launch<64, 2>(a, sh, st);
    return nt == 1 ? launch<128, 1>(a, sh, st) : launch<128, 2>(a, sh, st);
}

}  // namespace cp
