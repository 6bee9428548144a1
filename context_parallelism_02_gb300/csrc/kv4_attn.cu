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
// Codes are exact in fp16; q is scaled per row by a power of two into fp16's
// range (bf16's 8 bits fit), so the products are exact and the group's scale
// multiplies an fp32 sum.  The minima are one more product, m (fp16, exact) with
// the rows' group sums of q in three fp16 parts.  V's values s n + m are rounded
// to fp16 (relative 2^-11) and so are the weights P; the row sums are taken over
// the unrounded fp32 weights.
#include "kernels.h"
#include "kv4.cuh"
#include "tc_helpers.cuh"

namespace cp {

namespace {

constexpr float LN2 = 0.69314718055994530942f, LOG2E = 1.44269504088896340736f;
constexpr int WARPS = 4;

// D += A B, fp16 operands, fp32 accumulators, 16 x 8 x 16.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// The four code pairs of a word (nibbles e, e + 4 of the low and high half) as
// exact fp16 pairs: a nibble in the low bits of an fp16 of exponent 2^10 reads
// 1024 + n, in the next four bits 1024 + 16 n.
__device__ __forceinline__ void unpack(uint32_t w, __half2 (&n)[4])
{
    const __half2 k1024 = __float2half2_rn(1024.f), k16 = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.f);
    const uint32_t u = w >> 8;
    n[0] = __hsub2(as_h2((w & 0x000f000fu) | 0x64006400u), k1024);
    n[1] = __hfma2(as_h2((w & 0x00f000f0u) | 0x64006400u), k16, k64);
    n[2] = __hsub2(as_h2((u & 0x000f000fu) | 0x64006400u), k1024);
    n[3] = __hfma2(as_h2((u & 0x00f000f0u) | 0x64006400u), k16, k64);
}

__device__ __forceinline__ float ex2(float x) { return tc::ex2(x); }

// Query rows of one tile, as B operands, and what goes with a row.  Lane (g, c) =
// (lane / 4, lane % 4) holds row 8 t + g's share in q; the accumulators' columns
// are rows 8 t + 2c and 8 t + 2c + 1.
template <int D, int NT>
struct Rows {
    static constexpr int NG = Kv4<D>::NG;
    uint32_t q[NT][NG][4];     // group gr: elements 8 c + {0,1}, {2,3}, {4,5}, {6,7}
    uint32_t sum[NT][2];       // group c: hi, mid | lo, 0 of the sum of q
    float to_log2[NT][2];      // score -> log2 units, for the lane's two columns
    int limit[NT][2];          // slots that the column's row sees
    int min_limit, max_limit;  // over the tile
};

// Running state of a warp: m in log2 units (a lazily raised reference, not the
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
    it.h = i % Hkv;
    i /= Hkv;
    it.tile = i % s.tiles;
    it.j0 = i / s.tiles;
    return it;
}

template <int D, int NT>
__device__ __forceinline__ void load_rows(const Kv4AttnArgs &a, const Shape &sh, const Item &it, int len,
                                          Rows<D, NT> &r)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    int lo = 0x7fffffff, hi = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = (it.tile * NT + t) * 8 + g;
        const bool on = row < sh.rows;
        const int j = it.j0 + (on ? row / sh.group : 0);
        const int head = it.h * sh.group + (on ? row % sh.group : 0);
        uint4 w[NG];
        float top = 0.f;
        const uint4 *p = reinterpret_cast<const uint4 *>(a.q + (((int64_t)it.b * a.rows.n + j) * a.rows.Hq + head) * D);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            w[gr] = on ? __ldg(p + gr * 4 + c) : make_uint4(0, 0, 0, 0);
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
                const __half2 v = __floats2half2_rn(__uint_as_float(x[i] << 16) * up,
                                                    __uint_as_float(x[i] & 0xffff0000u) * up);
                r.q[t][gr][i] = h2(v);
                part += __low2float(v) + __high2float(v);
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
        const float back = a.scale * LOG2E / up;
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

// Scores of one block, in log2 units: x[t][0..1] token g, x[t][2..3] token g + 8.
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
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
        if (gr == c) na = ma[gr], nb = mb[gr];
    na = __byte_perm(na, na, 0x3232);
    nb = __byte_perm(nb, nb, 0x3232);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
        mma16816(x[t], na, nb, na, nb, r.sum[t][0], r.sum[t][1]);
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
        __half2 u[4], v[4];
        unpack(ka[gr], u);
        unpack(kb[gr], v);
        const float sa = __low2float(as_h2(ma[gr])), sb = __low2float(as_h2(mb[gr]));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(acc, h2(u[0]), h2(v[0]), h2(u[1]), h2(v[1]), r.q[t][gr][0], r.q[t][gr][1]);
            mma16816(acc, h2(u[2]), h2(v[2]), h2(u[3]), h2(v[3]), r.q[t][gr][2], r.q[t][gr][3]);
            x[t][0] = fmaf(sa, acc[0], x[t][0]);
            x[t][1] = fmaf(sa, acc[1], x[t][1]);
            x[t][2] = fmaf(sb, acc[2], x[t][2]);
            x[t][3] = fmaf(sb, acc[3], x[t][3]);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] *= r.to_log2[t][e & 1];
}

// Raises the references m where a score is more than 2^8 above them.
template <int D, int NT, int NB>
__device__ __forceinline__ void raise_max(const float (&x)[NB][NT][4], State<D, NT> &s)
{
    bool high = false;
    float top[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = -INFINITY;
#pragma unroll
            for (int i = 0; i < NB; ++i) v = fmaxf(v, fmaxf(x[i][t][e], x[i][t][e + 2]));
            top[t][e] = v;
            high |= v > s.m[t][e] + 8.f;
        }
    if (!__any_sync(0xffffffffu, high)) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = top[t][e];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            const float m = fmaxf(s.m[t][e], v);
            const float f = m == -INFINITY ? 1.f : ex2(s.m[t][e] - m);
            s.m[t][e] = m;
            s.l[t][e] *= f;
#pragma unroll
            for (int i = 0; i < 2 * Kv4<D>::NG; ++i) s.o[t][i][e] *= f, s.o[t][i][e + 2] *= f;
        }
}

// V^T fragments of group gr of a block: f[e][half], e = 0..3 the elements
// 32 gr + 4 g + e.  Tokens at or past `live` count as 0 whatever the block holds.
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

// O^T += V^T P^T for one block.  p: weights as B operands; live: tokens of the
// block whose values count (the others are taken as 0, codes and scales may be
// anything).
template <int D, int NT>
__device__ __forceinline__ void block_values(const uint8_t *blk, int live, const uint32_t (&p)[NT][2], State<D, NT> &s)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, c = lane & 3;
    uint32_t w[2][NG];
    uint2 sm[2][NG];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        load_words<NG>(blk + Kv4<D>::V_CODES + hf * 128 * NG + lane * 4 * NG, w[hf]);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
            sm[hf][gr] = *reinterpret_cast<const uint2 *>(blk + Kv4<D>::V_META + ((hf * 4 + c) * NG + gr) * 8);
        if (live < KV4_BLOCK) {
            const int k = hf * 8 + 2 * c;
            const uint32_t keep = (k < live ? 0x0000ffffu : 0u) | (k + 1 < live ? 0xffff0000u : 0u);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) sm[hf][gr].x &= keep, sm[hf][gr].y &= keep;
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
    }
}

// Whether a block's V scales or minima hold a value that is not finite.
template <int D>
__device__ __forceinline__ bool values_bad(const uint8_t *blk)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31;
    bool bad = false;
    for (int i = lane; i < 16 * NG; i += 32) {   // 16 NG words of two halves
        const uint32_t w = reinterpret_cast<const uint32_t *>(blk + Kv4<D>::V_META)[i];
        bad |= (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
    }
    return __any_sync(0xffffffffu, bad);
}

// One block of 16 tokens whose first slot is `slot`, for the warp's state.
template <int D, int NT>
__device__ __forceinline__ void block_step(const uint8_t *blk, int slot, const Rows<D, NT> &r, State<D, NT> &s)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float x[1][NT][4];
    block_scores<D, NT>(blk, r, x[0]);
    const bool cut = slot > r.min_limit - KV4_BLOCK;
    if (cut) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (slot + g + (e >> 1) * 8 >= r.limit[t][e & 1]) x[0][t][e] = -INFINITY;
    }
    raise_max<D, NT, 1>(x, s);
    uint32_t p[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float m = s.m[t][e & 1];
            w[e] = ex2(x[0][t][e] - (m == -INFINITY ? 0.f : m));
            s.l[t][e & 1] += w[e];
        }
        p[t][0] = movmatrix(h2(__floats2half2_rn(w[0], w[1])));
        p[t][1] = movmatrix(h2(__floats2half2_rn(w[2], w[3])));
    }
    const int live = r.max_limit - slot;
    if (cut && live > 0 && r.min_limit < r.max_limit && values_bad<D>(blk)) {
        // Rows see different tokens of this block and one of its values is not
        // finite: 0 times it would reach the rows that do not see it.  Row by row.
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
            uint32_t one[NT][2];
            int mine = 0;
#pragma unroll 1
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const int lim = __shfl_sync(0xffffffffu, (q & 1) ? r.limit[u][1] : r.limit[u][0], q >> 1);
                    if (u == t) mine = lim - slot;
                    one[u][0] = u == t && g == q ? p[u][0] : 0u;
                    one[u][1] = u == t && g == q ? p[u][1] : 0u;
                }
                State<D, NT> z;
                z.clear();
                block_values<D, NT>(blk, mine, one, z);
#pragma unroll
                for (int u = 0; u < NT; ++u)
#pragma unroll
                    for (int i = 0; i < 2 * Kv4<D>::NG; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (u == t && 2 * c + (e & 1) == q) s.o[u][i][e] += z.o[u][i][e];
            }
        }
        return;
    }
    block_values<D, NT>(blk, live, p, s);
}

// The warps' states of one item joined: rows' references and sums go through
// shared memory, then the accumulators are added up in the warps' order.
template <int D, int NT>
struct Joined {
    float m[WARPS][NT * 8], l[WARPS][NT * 8];
    float o[WARPS][NT * 8][D];
};

template <int D, int NT>
__device__ __forceinline__ void put_state(Joined<D, NT> &sm, const State<D, NT> &s)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = s.l[t][e];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (g == 0) {
                sm.m[warp][t * 8 + 2 * c + e] = s.m[t][e];
                sm.l[warp][t * 8 + 2 * c + e] = l;
            }
#pragma unroll
            for (int gr = 0; gr < Kv4<D>::NG; ++gr)
                *reinterpret_cast<float4 *>(&sm.o[warp][t * 8 + 2 * c + e][32 * gr + 4 * g]) =
                    make_float4(s.o[t][2 * gr][e], s.o[t][2 * gr][e + 2], s.o[t][2 * gr + 1][e], s.o[t][2 * gr + 1][e + 2]);
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(WARPS * 32) kv4_attn_kernel(Kv4AttnArgs a, Shape sh)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    Joined<D, NT> &sm = *reinterpret_cast<Joined<D, NT> *>(dyn);
    const int warp = threadIdx.x >> 5;
    const int b = blockIdx.x / sh.per_batch;
    const Item it = decode_item(sh, a.pool.Hkv, b, blockIdx.x % sh.per_batch);
    const int len = kv4_len(a.pool, b);
    Rows<D, NT> r;
    load_rows<D, NT>(a, sh, it, len, r);
    State<D, NT> s;
    s.clear();
    const int ps = a.pool.page_shift, bpp = 1 << (ps - 4);   // blocks per page
    const int32_t *sel = a.sel ? a.sel + (((int64_t)b * a.rows.n + it.j0) * a.pool.Hkv + it.h) * a.n_sel : nullptr;
    const int64_t blocks = sel ? (int64_t)a.n_sel * bpp : ((int64_t)r.max_limit + 15) >> 4;
    const int pages = (int)(((int64_t)len + (1 << ps) - 1) >> ps);
    for (int64_t i = warp; i < blocks; i += WARPS) {
        int lp = (int)(i >> (ps - 4));
        if (sel) {
            lp = __ldg(sel + lp);
            if (lp < 0) continue;
            if (lp >= pages) {
                kv4_report(a.pool.err);
                continue;
            }
        }
        const int slot = (lp << ps) + (int)(i & (bpp - 1)) * KV4_BLOCK;
        if (slot >= r.max_limit) continue;
        const int id = kv4_page(a.pool, b, lp);
        if (id < 0) continue;
        block_step<D, NT>(kv4_block<D>(a.pool, id, it.h, (int)(i & (bpp - 1))), slot, r, s);
    }
    put_state<D, NT>(sm, s);
    __syncthreads();
    for (int x = threadIdx.x; x < NT * 8 * (D / 4); x += WARPS * 32) {
        const int row = x / (D / 4), d4 = x % (D / 4);
        const int rr = it.tile * NT * 8 + row;
        if (rr >= sh.rows) continue;
        float m = -INFINITY;
        for (int w = 0; w < WARPS; ++w) m = fmaxf(m, sm.m[w][row]);
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < WARPS; ++w) {
            if (sm.m[w][row] == -INFINITY) continue;
            const float f = ex2(sm.m[w][row] - m);
            l = fmaf(f, sm.l[w][row], l);
            const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][row][d4 * 4]);
            o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
        }
        const int j = it.j0 + rr / sh.group, head = it.h * sh.group + rr % sh.group;
        const bool empty = l == 0.f;
        const float inv = empty ? 0.f : 1.f / l;
        o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
        const int64_t at = (((int64_t)b * a.rows.n + j) * a.rows.Hq + head) * D + d4 * 4;
        if (a.out_f32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = o;
        } else {
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
                make_uint2(tc::pack_bf16(o.x, o.y), tc::pack_bf16(o.z, o.w));
        }
        if (d4 == 0) a.lse[((int64_t)b * a.rows.Hq + head) * a.rows.n + j] = empty ? -INFINITY : fmaf(m, LN2, logf(l));
    }
}

template <int D, int NT>
int launch(const Kv4AttnArgs &a, const Shape &sh, cudaStream_t st)
{
    const int64_t items = (int64_t)a.rows.B * sh.per_batch;
    if (items > 0x7fffffffLL) return CP_EUNSUPPORTED;
    constexpr int smem = sizeof(Joined<D, NT>);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kv4_attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return CP_ECUDA;
    kv4_attn_kernel<D, NT><<<(unsigned)items, WARPS * 32, smem, st>>>(a, sh);
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace

size_t kv4_attn_workspace_bytes(int D) { return D == 64 || D == 128 ? 256 : 0; }

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
