// kv4_append.cu -- writing tokens into the paged 4-bit cache (rotation and
// quantisation on the way) and reading slots back.
//
// Rotation of a pair (x1, x2) by the angle of its position:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin,
// in fp32 with every product and sum rounded by itself.  Quantisation of a
// group of 32 elements of a row: s = fp16((max - min) fp32(1/15)), m = fp16(min),
// code = clamp(rint((y - m) / s), 0, 15); a group with a value that is not
// finite is held as NaN.
//
// Per token and kv head 2 D elements are read and 1.25 D bytes written.  The q rows are
// bound by that traffic; the k and v rows are not: the quantisation takes about 600
// instructions for the K and V rows of two tokens and a head, in one dependent chain a
// pass.  32768 tokens of 8 kv and 32 q heads take 151 us, 713 MB at 4.7 TB/s: 66 % of the
// issue slots, 59 % of DRAM, and warps that mostly wait for their rows (4.2 of 10 cycles a
// warp and instruction); the k and v rows alone 84 to 96 us, of which their bytes
// are 26, the q rows alone 92.
// In K and V a lane holds 8 neighbouring elements of a row, so a group's extremes are
// two shuffles and a K code word is one lane's; a warp's pass takes the K rows of
// 256 / D tokens, the next their V rows (one pass over both left lanes idle in the
// rotation: 387 us against 347 at that stage).  Blocks of 16 tokens that are written
// whole are put together in shared memory and leave in 16-byte pieces.  q rows: all
// heads of a token per warp, so that a row of the tables is read once for them.
#include "kernels.h"
#include "kv4.cuh"

namespace cp {

namespace {

__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// 8 elements as they are in memory
struct Raw16 { uint4 a; };
struct Raw32 { float4 a, b; };
__device__ __forceinline__ void fetch8(const __nv_bfloat16 *p, Raw16 &r) { r.a = *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void fetch8(const float *p, Raw32 &r)
{
    r.a = reinterpret_cast<const float4 *>(p)[0];
    r.b = reinterpret_cast<const float4 *>(p)[1];
}
__device__ __forceinline__ void clear(Raw16 &r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void clear(Raw32 &r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void widen(const Raw16 &r, float (&x)[8])
{
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(const Raw32 &r, float (&x)[8])
{
    x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
    x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
template <typename T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { using type = Raw16; };
template <> struct RawOf<float> { using type = Raw32; };

// 4 elements of a q row
__device__ __forceinline__ void load4(const float *p, float (&x)[4])
{
    const float4 a = *reinterpret_cast<const float4 *>(p);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4])
{
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(a.x << 16), x[1] = __uint_as_float(a.x & 0xffff0000u);
    x[2] = __uint_as_float(a.y << 16), x[3] = __uint_as_float(a.y & 0xffff0000u);
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void store4(float *p, const float (&x)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&x)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}

// Rotates the 8 elements d0.. of a row spread over consecutive lanes (8 per
// lane).  Every lane of the warp calls it; lanes with turn == false keep x.
template <bool INTER>
__device__ __forceinline__ void rotate8(float (&x)[8], const Kv4AppendArgs &a, int d0, int pos, bool turn)
{
    const int half = a.rot >> 1;
    const bool in = turn && d0 < a.rot;
    if (INTER) {
        if (in) {
            const int64_t at = (int64_t)pos * half + (d0 >> 1);
            const float4 cv = *reinterpret_cast<const float4 *>(a.cos + at);
            const float4 sv = *reinterpret_cast<const float4 *>(a.sin + at);
            const float cs[4] = {cv.x, cv.y, cv.z, cv.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x1 = x[2 * i], x2 = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(x1, cs[i]), __fmul_rn(x2, sn[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(x2, cs[i]), __fmul_rn(x1, sn[i]));
            }
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const bool first = d0 < half;
    const int src = in ? (first ? lane + (half >> 3) : lane - (half >> 3)) : lane;
    const float sign = first ? -1.f : 1.f;   // x1 cos - x2 sin, x2 cos + x1 sin
    float cs[8], sn[8];
    if (in) {
        const int64_t at = (int64_t)pos * half + (first ? d0 : d0 - half);
        load8(a.cos + at, cs);
        load8(a.sin + at, sn);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = __shfl_sync(0xffffffffu, x[i], src);
        if (in) x[i] = __fadd_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(p, sign * sn[i]));
    }
}

// Position of token (b, j); -1 (and CP_ECACHE) outside the rotation table, 0 where
// nothing is rotated.
__device__ __forceinline__ int position(const Kv4AppendArgs &a, int b, int j, int64_t slot)
{
    if (!a.rot) return 0;
    const int64_t p = a.positions ? (int64_t)a.positions[(int64_t)b * a.n + j] : slot;
    if (p < 0 || p >= a.max_pos) {
        kv4_report(a.pool.err);
        return -1;
    }
    return (int)p;
}

__device__ __forceinline__ int new_tokens(const Kv4AppendArgs &a, int b)
{
    if (!a.n_new) return a.n;
    const int m = a.n_new[b];
    return m < 0 ? 0 : m > a.n ? a.n : m;
}

// Largest magnitude that is kept: with the roundings of s (half a step of 8, 15
// times) and m (half of 32) on top, s code + m still rounds to a finite fp16.
constexpr float KV4_MAX = 65408.f;

// min and max of three that keep a NaN
__device__ __forceinline__ float min3(float a, float b, float c)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One code by division (out of line: eight divisions are a lot of code).
__device__ __noinline__ float code_by_division(float y, float s)
{
    return s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(y, s)), 0.f), 15.f) : 0.f;
}

// Codes (as whole floats), scale and minimum of a lane's 8 elements; the group is
// 4 lanes.  s is the range times fp32(1 / 15).  rint((y - m) / s) is taken from
// 15 clamp((y - m) a, 0, 1) with a = fp32(1 / s) fp32(1 / 15): one reciprocal a group,
// the clamp is the product's own, the rounding that of adding 1.5 2^23.  The factors
// are off by 2.5 units in the last place together and the quotient by a half:
// 15 (2.5 2^-23 + 2^-24) < 6e-6.  Where a lane's product comes within 1e-5 of a half the
// warp divides: bf16 values sit on exact halves of s often enough (4 in 10^4 elements)
// that the nearest-even rule of the quotient has to hold for them.
__device__ __forceinline__ void quantise8(const float (&x)[8], float (&code)[8], __half &s, __half &m)
{
    float lo = min3(min3(x[0], x[1], x[2]), min3(x[3], x[4], x[5]), min3(x[6], x[7], x[7]));
    float hi = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
    {
        const float l1 = __shfl_xor_sync(0xffffffffu, lo, 1), h1 = __shfl_xor_sync(0xffffffffu, hi, 1);
        lo = min3(lo, l1, l1);
        hi = max3(hi, h1, h1);
        const float l2 = __shfl_xor_sync(0xffffffffu, lo, 2), h2 = __shfl_xor_sync(0xffffffffu, hi, 2);
        lo = min3(lo, l2, l2);
        hi = max3(hi, h2, h2);
    }
    const bool bad = !(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY);
    // beyond the largest magnitude: an element's code comes out as its clamped value's
    lo = fminf(fmaxf(lo, -KV4_MAX), KV4_MAX);
    hi = fminf(fmaxf(hi, -KV4_MAX), KV4_MAX);
    constexpr float FIFTEENTH = 1.f / 15.f;
    s = __float2half_rn(__fmul_rn(hi - lo, FIFTEENTH));
    m = __float2half_rn(lo);
    const float sf = __half2float(s), mf = __half2float(m);
    const float a = sf > 0.f && !bad ? __fmul_rn(__frcp_rn(sf), FIFTEENTH) : 0.f;   // 0: every code is 0
    if (bad) s = __ushort_as_half(0), m = __ushort_as_half(0x7fff);
    constexpr float ROUND = 12582912.f;
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float u;
        asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(u) : "f"(__fsub_rn(x[i], mf)), "f"(a));
        code[i] = __fsub_rn(__fmaf_rn(u, 15.f, ROUND), ROUND);
        off = fmaxf(off, fabsf(__fmaf_rn(u, 15.f, -code[i])));
    }
    if (__any_sync(0xffffffffu, off > 0.49999f)) {
        if (off > 0.49999f) {   // a is 0 where the group is constant or not finite: not here
#pragma unroll
            for (int i = 0; i < 8; ++i)
                code[i] = code_by_division(__fsub_rn(fminf(fmaxf(x[i], -KV4_MAX), KV4_MAX), mf), sf);
        }
    }
}

// Four codes as the nibbles of the low 16 bits (what is above them is 2^23's).
__device__ __forceinline__ uint32_t nibbles(float a, float b, float c, float d)
{
    return __float_as_uint(fmaf(fmaf(fmaf(d, 16.f, c), 16.f, b), 16.f, a) + 8388608.f);
}

// Bytes of a V code word and of its scale for token t, group gr.
template <int D>
__device__ __forceinline__ int v_code_at(int t, int gr, int g)
{
    constexpr int NG = Kv4<D>::NG;
    return Kv4<D>::V_CODES + ((t >> 3) * 32 * NG + (4 * g + ((t & 7) >> 1)) * NG + gr) * 4 + (t & 1) * 2;
}
template <int D>
__device__ __forceinline__ int v_meta_at(int t, int gr)
{
    return Kv4<D>::V_META + (((t >> 3) * 4 + ((t & 7) >> 1)) * Kv4<D>::NG + gr) * 8 + (t & 1) * 2;
}

// A warp's q rows: `span` eights of heads of one token.  A lane holds 4 + 4 elements
// of a row: the two halves of 4 pairs, 4 pairs that lie together (interleaved), or 8
// elements that are not rotated.
template <int D, typename T, bool INTER>
__device__ __forceinline__ void rotate_q(const Kv4AppendArgs &a, unsigned unit, int span, int spans)
{
    constexpr int LPR = D / 8, RPP = 32 / LPR, U = 8 / RPP;   // lanes of a row, rows of a pass, passes
    const int lane = threadIdx.x & 31, l = lane & (LPR - 1);
    const unsigned bj = unit / (unsigned)spans;
    const int first = (int)(unit - bj * spans) * span * 8;
    const int b = (int)(bj / (unsigned)a.n), j = (int)(bj - (unsigned)b * a.n);
    const bool real = j < new_tokens(a, b);
    const int pos = real ? position(a, b, j, (int64_t)a.pool.lens[b] + j) : -1;
    const bool on = pos >= 0;                       // rows that are not there, or have no angle, are 0
    const bool turn = on && 8 * l < a.rot;
    int da = 8 * l, db = 8 * l + 4;
    if (!INTER && 8 * l < a.rot) da = 4 * l, db = 4 * l + (a.rot >> 1);
    float cs[4], sn[4];
    if (turn) {
        const float4 cv = *reinterpret_cast<const float4 *>(a.cos + (int64_t)pos * (a.rot >> 1) + 4 * l);
        const float4 sv = *reinterpret_cast<const float4 *>(a.sin + (int64_t)pos * (a.rot >> 1) + 4 * l);
        cs[0] = cv.x, cs[1] = cv.y, cs[2] = cv.z, cs[3] = cv.w;
        sn[0] = sv.x, sn[1] = sv.y, sn[2] = sv.z, sn[3] = sv.w;
    }
    const T *p = static_cast<const T *>(a.q) + b * a.qs[0] + j * a.qs[1] + (first + lane / LPR) * a.qs[2];
    T *to = static_cast<T *>(a.q_out) + ((int64_t)bj * a.Hq + first + lane / LPR) * D;
    const int64_t step = RPP * a.qs[2];
    const int last = min(first + span * 8, a.Hq);
#pragma unroll 1
    for (int h0 = first + lane / LPR; h0 - lane / LPR < last; h0 += 8) {
        float x[U][4], y[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = y[u][i] = 0.f;
            if (on && h0 + u * RPP < last) {
                load4(p + u * step + da, x[u]);
                load4(p + u * step + db, y[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * RPP >= last) break;
            if (turn) {
                // pairs (x[i], y[i]), or (x[0], x[1]), (x[2], x[3]), (y[0], y[1]), (y[2], y[3])
                float r[8] = {x[u][0], x[u][1], x[u][2], x[u][3], y[u][0], y[u][1], y[u][2], y[u][3]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float &x1 = INTER ? r[2 * i] : r[i], &x2 = INTER ? r[2 * i + 1] : r[4 + i];
                    const float r1 = __fsub_rn(__fmul_rn(x1, cs[i]), __fmul_rn(x2, sn[i]));
                    const float r2 = __fadd_rn(__fmul_rn(x2, cs[i]), __fmul_rn(x1, sn[i]));
                    x1 = r1;
                    x2 = r2;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = r[i], y[u][i] = r[4 + i];
            }
            store4(to + u * RPP * D + da, x[u]);
            store4(to + u * RPP * D + db, y[u]);
        }
        p += U * step;
        to += 8 * D;
    }
}

// A warp's pass over tokens of K rows (8 elements a lane): rotated, taken into the
// elements' extremes (bf16 pairs), quantised and written to `to`.
template <int D, bool INTER>
__device__ __forceinline__ void k_pass(float (&x)[8], const Kv4AppendArgs &a, int t, int pos, bool on, uint8_t *to,
                                       __nv_bfloat162 (&lo)[4], __nv_bfloat162 (&hi)[4])
{
    constexpr int NG = Kv4<D>::NG;
    const int sub = threadIdx.x & (D / 8 - 1), gr = sub >> 2, q4 = sub & 3;
    if (a.rot) rotate8<INTER>(x, a, sub * 8, pos, on);
    if (a.summary && on) {
        const float size = fabsf(x[0]) + fabsf(x[1]) + fabsf(x[2]) + fabsf(x[3]) + fabsf(x[4]) + fabsf(x[5]) + fabsf(x[6]) +
                           fabsf(x[7]);
        __nv_bfloat162 v[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        if (__any_sync(__activemask(), !(size < INFINITY))) {   // a key that is not finite opens its element's range
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!isfinite(x[2 * i])) v[i].x = __float2bfloat16_rn(-INFINITY), w[i].x = __float2bfloat16_rn(INFINITY);
                if (!isfinite(x[2 * i + 1])) v[i].y = __float2bfloat16_rn(-INFINITY), w[i].y = __float2bfloat16_rn(INFINITY);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __hmin2(lo[i], v[i]);
            hi[i] = __hmax2(hi[i], w[i]);
        }
    }
    float code[8];
    __half s, m;
    quantise8(x, code, s, m);
    if (!on) return;
    *reinterpret_cast<uint32_t *>(to + t * (D / 2) + (q4 * NG + gr) * 4) =
        __byte_perm(nibbles(code[0], code[2], code[4], code[6]), nibbles(code[1], code[3], code[5], code[7]), 0x5410);
    if (q4 == 0) *reinterpret_cast<__half2 *>(to + Kv4<D>::K_META + (t * NG + gr) * 4) = __halves2half2(s, m);
}

template <int D>
__device__ __forceinline__ void v_pass(const float (&x)[8], int t, bool on, uint8_t *to)
{
    const int sub = threadIdx.x & (D / 8 - 1), gr = sub >> 2, q4 = sub & 3;
    float code[8];
    __half s, m;
    quantise8(x, code, s, m);
    if (!on) return;
#pragma unroll
    for (int e = 0; e < 2; ++e)
        *reinterpret_cast<uint16_t *>(to + v_code_at<D>(t, gr, 2 * q4 + e)) =
            (uint16_t)nibbles(code[4 * e], code[4 * e + 1], code[4 * e + 2], code[4 * e + 3]);
    if (q4 == 0) {
        uint8_t *p = to + v_meta_at<D>(t, gr);
        *reinterpret_cast<__half *>(p) = s;
        *reinterpret_cast<__half *>(p + 4) = m;
    }
}

// Four warps.  kv_blocks of the grid's blocks take (chunk of max(page, 64) slots,
// kv head) of a sequence each, a warp 16 slots of it at a time; the others q rows.
// The two kinds alternate (every `every`-th block is a kv block), so that the
// arithmetic of one and the memory traffic of the other share an SM.
template <int D, typename T, bool INTER>
__global__ void __launch_bounds__(128, 7) kv4_append_kernel(Kv4AppendArgs a, int chunk_shift, unsigned chunks, unsigned kv_blocks,
                                                         unsigned q_units, int span, int spans, unsigned every)
{
    constexpr int LPR = D / 8;           // lanes of a row
    constexpr int TPP = 32 / LPR;        // tokens of a pass
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // kv blocks at multiples of `every`, as long as there are any (32-bit indices: a
    // 64-bit division is a hundred instructions, as much as a q row's work)
    kv4_begin();
    const unsigned bid = blockIdx.x, kb = bid / every;
    if (kb * every != bid || kb >= kv_blocks) {
        const unsigned before = min(kb + 1, kv_blocks);   // kv blocks in front
        const unsigned unit = (bid - before) * 4 + warp;
        if (unit < q_units) rotate_q<D, T, INTER>(a, unit, span, spans);
        return;
    }
    __shared__ __nv_bfloat16 red[4][2][D];
    __shared__ __align__(16) uint8_t stage[4][Kv4<D>::BYTES];
    const int sub = lane & (LPR - 1), d0 = sub * 8, tsub = lane / LPR;
    const unsigned bc = kb / (unsigned)a.pool.Hkv;
    const int h = (int)(kb - bc * a.pool.Hkv), b = (int)(bc / chunks), c = (int)(bc - b * chunks);
    const int64_t len = a.pool.lens[b];
    if (len < 0) {
        if (threadIdx.x == 0) kv4_report(a.pool.err);
        return;
    }
    const int64_t end = len + new_tokens(a, b);
    const int64_t c0 = ((len >> chunk_shift) + c) << chunk_shift;   // first slot of the chunk
    if (c0 >= end) return;
    const int chunk = 1 << chunk_shift;
    const int ps = a.pool.page_shift;
    const T *const k0 = static_cast<const T *>(a.k) + b * a.ks[0] + h * a.ks[2] + d0;
    const T *const v0 = static_cast<const T *>(a.v) + b * a.vs[0] + h * a.vs[2] + d0;
    __nv_bfloat162 lo[4], hi[4];   // extremes of the K rows that this lane has seen
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = __float2bfloat162_rn(INFINITY), hi[i] = __float2bfloat162_rn(-INFINITY);
    for (int s0 = warp * KV4_BLOCK; s0 < chunk; s0 += 4 * KV4_BLOCK) {
        const int64_t slot0 = c0 + s0;
        if (slot0 >= end || slot0 + KV4_BLOCK <= len) continue;
        const int id = kv4_page(a.pool, b, slot0 >> ps);
        if (id < 0) continue;
        uint8_t *const blk = kv4_block<D>(a.pool, id, h, (int)((slot0 & ((1 << ps) - 1)) >> 4));
        const int t_lo = len > slot0 ? (int)(len - slot0) : 0;
        const int t_hi = end - slot0 < KV4_BLOCK ? (int)(end - slot0) : KV4_BLOCK;
        // lane t: whether token t is written, and its position
        const bool mine = lane >= t_lo && lane < t_hi;
        const int at = mine ? position(a, b, (int)(slot0 + lane - len), slot0 + lane) : -1;
        const unsigned live = __ballot_sync(0xffffffffu, at >= 0);
        const bool full = live == 0xffffu;
        uint8_t *const to = full ? stage[warp] : blk;
        int t = t_lo + tsub;
        const T *kp = k0 + (slot0 + t - len) * a.ks[1], *vp = v0 + (slot0 + t - len) * a.vs[1];
        typename RawOf<T>::type kr, vr;      // the next pass's rows, on their way during this one
        clear(kr);
        clear(vr);
        if (live >> t & 1) {                 // t < 32
            fetch8(kp, kr);
            fetch8(vp, vr);
        }
#pragma unroll 1
        for (int t0 = t_lo; t0 < t_hi; t0 += TPP, t += TPP) {
            const bool on = live >> t & 1;
            const int pos = __shfl_sync(0xffffffffu, at, t);
            const bool more = t + TPP < KV4_BLOCK && (live >> (t + TPP) & 1);
            float x[8];
            widen(kr, x);
            kp += TPP * a.ks[1];
            if (more) fetch8(kp, kr);
            k_pass<D, INTER>(x, a, t, pos, on, to, lo, hi);
            widen(vr, x);
            vp += TPP * a.vs[1];
            if (more) fetch8(vp, vr);
            v_pass<D>(x, t, on, to);
        }
        __syncwarp();
        if (full) {
#pragma unroll
            for (int i = 0; i < Kv4<D>::BYTES / 512; ++i)
                reinterpret_cast<uint4 *>(blk)[i * 32 + lane] = reinterpret_cast<const uint4 *>(stage[warp])[i * 32 + lane];
            if (Kv4<D>::BYTES % 512 && lane < Kv4<D>::BYTES % 512 / 16)
                reinterpret_cast<uint4 *>(blk)[Kv4<D>::BYTES / 512 * 32 + lane] =
                    reinterpret_cast<const uint4 *>(stage[warp])[Kv4<D>::BYTES / 512 * 32 + lane];
            __syncwarp();
        }
    }
    if (!a.summary) return;
    // extremes over the lanes that hold the same elements of other tokens, then over
    // the warps that share a page
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
            lo[i] = __hmin2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
            hi[i] = __hmax2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        }
        if (tsub == 0) {
            *reinterpret_cast<__nv_bfloat162 *>(&red[warp][0][d0 + 2 * i]) = lo[i];
            *reinterpret_cast<__nv_bfloat162 *>(&red[warp][1][d0 + 2 * i]) = hi[i];
        }
    }
    __syncthreads();
    const int share = (1 << ps) >= 64 ? 4 : (1 << ps) / KV4_BLOCK;   // warps that share a page
    for (int x = threadIdx.x; x < (4 / share) * 2 * D; x += 128) {
        const int p = x / (2 * D), mx = x / D & 1, d = x % D;
        const int64_t p0 = c0 + ((int64_t)p << ps);   // first slot of the page
        if (p0 >= end || p0 + (1 << ps) <= len) continue;
        __nv_bfloat16 r = red[p * share][mx][d];
        for (int w = 1; w < share; ++w) r = mx ? __hmax(r, red[p * share + w][mx][d]) : __hmin(r, red[p * share + w][mx][d]);
        const int id = kv4_page(a.pool, b, p0 >> ps);
        if (id < 0) continue;
        __nv_bfloat16 *to = a.summary + (((int64_t)id * a.pool.Hkv + h) * 2 + mx) * D + d;
        if (p0 < len) r = mx ? __hmax(r, *to) : __hmin(r, *to);
        *to = r;
    }
}

// One warp per 16-token block and kv head.  Lane (g, c) = (lane / 4, lane % 4)
// takes the words that lie together for it: of K, elements 8 c .. 8 c + 7 of every
// group of tokens g and g + 8; of V, elements 4 g .. 4 g + 3 of every group of
// tokens 2 c, 2 c + 1, 8 + 2 c and 9 + 2 c.  All loads are 16 bytes (D = 128) and on
// their way before the first is used; stores cover 64 bytes of a row or more.
template <int N>
__device__ __forceinline__ void words(const uint8_t *p, uint32_t (&w)[N])
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

__device__ __forceinline__ float half_of(uint32_t w, int hi)
{
    return __half2float(__ushort_as_half((unsigned short)(hi ? w >> 16 : w & 0xffffu)));
}

template <int D, typename T>
__global__ void __launch_bounds__(128) kv4_gather_kernel(Kv4GatherArgs a, unsigned blocks, unsigned warps)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const unsigned wid = blockIdx.x * 4 + (threadIdx.x >> 5);
    kv4_begin();
    if (wid >= warps) return;
    // heads next to each other: their rows are neighbours in k and v
    const unsigned bx = wid / (unsigned)a.pool.Hkv;
    const int h = (int)(wid - bx * a.pool.Hkv), b = (int)(bx / blocks), x = (int)(bx - b * blocks);
    const int len = kv4_len(a.pool, b);
    int64_t first = a.start ? (int64_t)a.start[b] : 0;
    if (first < 0) {
        if (lane == 0) kv4_report(a.pool.err);
        first = len;   // no slot to read: every row is written as 0
    }
    const int64_t slot0 = ((first >> 4) + x) << 4;
    const int ps = a.pool.page_shift;
    uint32_t k[2][NG], km[2][NG], v[2][NG], vm[2][2 * NG];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) k[i][gr] = km[i][gr] = v[i][gr] = vm[i][gr] = vm[i][NG + gr] = 0;
    }
    if (slot0 < len && slot0 < first + a.count) {
        const int id = kv4_page(a.pool, b, slot0 >> ps);
        if (id >= 0) {
            const uint8_t *blk = kv4_block<D>(a.pool, id, h, (int)((slot0 & ((1 << ps) - 1)) >> 4));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                words<NG>(blk + (g + 8 * i) * (D / 2) + c * 4 * NG, k[i]);
                words<NG>(blk + Kv4<D>::K_META + (g + 8 * i) * 4 * NG, km[i]);
                words<NG>(blk + Kv4<D>::V_CODES + i * 128 * NG + lane * 4 * NG, v[i]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t part[NG];
                    words<NG>(blk + Kv4<D>::V_META + ((i * 4 + c) * 2 + y) * 4 * NG, part);
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) vm[i][y * NG + gr] = part[gr];
                }
            }
        }
    }
    const int64_t row0 = (int64_t)b * a.count;
    const int64_t live = len - slot0;   // tokens of the block below the length; the others are written as 0
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = g + 8 * i;
        const int64_t j = slot0 + t - first;
        if (j < 0 || j >= a.count) continue;
        T *to = static_cast<T *>(a.k) + ((row0 + j) * a.pool.Hkv + h) * D + 8 * c;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            const float s = half_of(km[i][gr], 0), m = half_of(km[i][gr], 1);
            float y[8];
#pragma unroll
            for (int o = 0; o < 8; ++o) {
                const int code = k[i][gr] >> (4 * ((o >> 1) + 4 * (o & 1))) & 15;
                y[o] = t < live ? __fadd_rn(__fmul_rn((float)code, s), m) : 0.f;
            }
            store8(to + 32 * gr, y);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int lo = 0; lo < 2; ++lo) {
            const int t = 8 * i + 2 * c + lo;
            const int64_t j = slot0 + t - first;
            if (j < 0 || j >= a.count) continue;
            T *to = static_cast<T *>(a.v) + ((row0 + j) * a.pool.Hkv + h) * D + 4 * g;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                const float s = half_of(vm[i][2 * gr], lo), m = half_of(vm[i][2 * gr + 1], lo);
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int code = v[i][gr] >> (16 * lo + 4 * e) & 15;
                    y[e] = t < live ? __fadd_rn(__fmul_rn((float)code, s), m) : 0.f;
                }
                store4(to + 32 * gr, y);
            }
        }
}

}  // namespace

int launch_kv4_append(const Kv4AppendArgs &a, int D, int dtype, cudaStream_t st)
{
    const int chunk_shift = a.pool.page_shift > 6 ? a.pool.page_shift : 6;
    const int chunk = 1 << chunk_shift;
    const int64_t chunks = ((int64_t)a.n + chunk - 2) / chunk + 1;
    const int64_t kv_blocks = chunks * a.pool.Hkv * a.B;
    // q: a warp takes all heads of a token where there are tokens enough to fill the
    // GPU, else eight
    const int64_t tokens = (int64_t)a.B * a.n;
    const int eights = (a.Hq + 7) / 8;
    const int span = tokens >= (int64_t)sm_count() * 32 ? eights : 1, spans = (eights + span - 1) / span;
    const int64_t q_units = a.q ? tokens * spans : 0;
    const int64_t blocks = kv_blocks + (q_units + 3) / 4;
    if (blocks > 0x3fffffffLL || q_units > 0x7fffffffLL) return CP_EUNSUPPORTED;
    const unsigned every = (unsigned)(blocks / kv_blocks);
    cudaError_t rc;
#define CP_KV4_LAUNCH(D_, T_, I_)                                                                                     \
    rc = kv4_launch(kv4_append_kernel<D_, T_, I_>, (unsigned)blocks, 128, 0, st, a, chunk_shift, (unsigned)chunks,    \
                    (unsigned)kv_blocks, (unsigned)q_units, span, spans, every)
#define CP_KV4_APPEND(D_, T_)                          \
    do {                                               \
        if (a.interleaved) CP_KV4_LAUNCH(D_, T_, true); \
        else CP_KV4_LAUNCH(D_, T_, false);             \
    } while (0)
    if (D == 64) {
        if (dtype == CP_BF16) CP_KV4_APPEND(64, __nv_bfloat16);
        else CP_KV4_APPEND(64, float);
    } else {
        if (dtype == CP_BF16) CP_KV4_APPEND(128, __nv_bfloat16);
        else CP_KV4_APPEND(128, float);
    }
#undef CP_KV4_APPEND
#undef CP_KV4_LAUNCH
    return rc == cudaSuccess ? CP_OK : CP_ECUDA;
}

int launch_kv4_gather(const Kv4GatherArgs &a, int D, int dtype, cudaStream_t st)
{
    // an unaligned start reaches one block more
    const int64_t blocks = ((int64_t)a.count + KV4_BLOCK - 2) / KV4_BLOCK + 1;
    const int64_t warps = blocks * a.pool.Hkv * a.B;
    const int64_t grid = (warps + 3) / 4;
    if (warps > 0x7fffffffLL) return CP_EUNSUPPORTED;
    cudaError_t rc;
#define CP_KV4_GATHER(D_, T_) \
    rc = kv4_launch(kv4_gather_kernel<D_, T_>, (unsigned)grid, 128, 0, st, a, (unsigned)blocks, (unsigned)warps)
    if (D == 64) {
        if (dtype == CP_BF16) CP_KV4_GATHER(64, __nv_bfloat16);
        else CP_KV4_GATHER(64, float);
    } else {
        if (dtype == CP_BF16) CP_KV4_GATHER(128, __nv_bfloat16);
        else CP_KV4_GATHER(128, float);
    }
#undef CP_KV4_GATHER
    return rc == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace cp
