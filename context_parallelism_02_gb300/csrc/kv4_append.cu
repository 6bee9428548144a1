// kv4_append.cu -- writing tokens into the paged 4-bit cache (rotation and
// quantisation on the way) and reading slots back.
//
// Rotation of a pair (x1, x2) by the angle of its position:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin,
// in fp32 with every product and sum rounded by itself.  Quantisation of a
// group of 32 elements of a row: s = fp16((max - min) / 15), m = fp16(min),
// code = clamp(rint((y - m) / s), 0, 15); a group with a value that is not
// finite is held as NaN.
//
// HBM-bound: per token and kv head 2 D elements are read and 1.25 D bytes
// written.  A lane holds 8 neighbouring elements of a row, so a group's extremes
// are two shuffles and a K code word is one lane's.  K and V rows of a token sit
// in one warp (a decode step, one token per sequence, is one pass of one warp).
#include "kernels.h"
#include "kv4.cuh"

namespace cp {

namespace {

__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8])
{
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
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

// Rotates the 8 elements d0.. of a row spread over consecutive lanes (8 per
// lane).  Every lane of the warp calls it; lanes with turn == false keep x.
__device__ __forceinline__ void rotate8(float (&x)[8], const Kv4AppendArgs &a, int d0, int64_t pos, bool turn)
{
    const int half = a.rot >> 1;
    const int lane = threadIdx.x & 31;
    if (a.interleaved) {
        if (turn && d0 < a.rot) {
            const int64_t at = pos * half + (d0 >> 1);
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
    const bool in = turn && d0 < a.rot;
    const bool first = d0 < half;
    const int src = in ? (first ? lane + (half >> 3) : lane - (half >> 3)) : lane;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], src);
    if (in) {
        float cs[8], sn[8];
        const int64_t at = pos * half + (first ? d0 : d0 - half);
        load8(a.cos + at, cs);
        load8(a.sin + at, sn);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __fmul_rn(x[i], cs[i]), w = __fmul_rn(p[i], sn[i]);
            x[i] = first ? __fsub_rn(u, w) : __fadd_rn(u, w);
        }
    }
}

// Position of token (b, j); -1 (and CP_ECACHE) outside the rotation table.
__device__ __forceinline__ int64_t position(const Kv4AppendArgs &a, int b, int j, int64_t slot)
{
    const int64_t p = a.positions ? (int64_t)__ldg(a.positions + (int64_t)b * a.n + j) : slot;
    if (a.rot && (p < 0 || p >= a.max_pos)) {
        kv4_report(a.pool.err);
        return -1;
    }
    return p;
}

__device__ __forceinline__ int new_tokens(const Kv4AppendArgs &a, int b)
{
    if (!a.n_new) return a.n;
    const int m = __ldg(a.n_new + b);
    return m < 0 ? 0 : m > a.n ? a.n : m;
}

// Largest magnitude that is kept: with the roundings of s (half a step of 8, 15
// times) and m (half of 32) on top, s code + m still rounds to a finite fp16.
constexpr float KV4_MAX = 65408.f;

// Codes, scale and minimum of a lane's 8 elements; the group is 4 lanes.
__device__ __forceinline__ void quantise8(const float (&x)[8], int (&code)[8], __half &s, __half &m)
{
    bool bad = false;
    float y[8], lo, hi;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bad |= !isfinite(x[i]);
        y[i] = fminf(fmaxf(x[i], -KV4_MAX), KV4_MAX);
        lo = i ? fminf(lo, y[i]) : y[i];
        hi = i ? fmaxf(hi, y[i]) : y[i];
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const unsigned group = 0xfu << (threadIdx.x & 28);
    bad = (__ballot_sync(0xffffffffu, bad) & group) != 0;
    s = __float2half_rn(bad ? 0.f : __fdiv_rn(hi - lo, 15.f));
    m = bad ? __ushort_as_half(0x7fff) : __float2half_rn(lo);
    const float sf = __half2float(s), mf = __half2float(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = sf > 0.f ? rintf(__fdiv_rn(y[i] - mf, sf)) : 0.f;
        code[i] = (int)fminf(fmaxf(t, 0.f), 15.f);
    }
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

// Warps of a block: 4.  The first kv_blocks blocks take (batch, kv head, chunk
// of max(page, 64) slots), the others 128 / (D / 8) rows of q each.
template <int D, typename T>
__global__ void __launch_bounds__(128) kv4_append_kernel(Kv4AppendArgs a, int chunk_shift, int chunks, int64_t kv_blocks)
{
    constexpr int LPR = D / 8;           // lanes of a row
    constexpr int TPI = 16 / LPR;        // tokens of a warp's pass (K and V rows)
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & (LPR - 1), d0 = sub * 8;
    if ((int64_t)blockIdx.x >= kv_blocks) {   // q rows
        const int64_t row = ((int64_t)blockIdx.x - kv_blocks) * (128 / LPR) + threadIdx.x / LPR;
        const int64_t rows = (int64_t)a.B * a.n * a.Hq;
        const bool on = row < rows;
        const int h = on ? (int)(row % a.Hq) : 0;
        const int64_t bj = on ? row / a.Hq : 0;
        const int j = (int)(bj % a.n), b = (int)(bj / a.n);
        const bool real = on && j < new_tokens(a, b);
        const int64_t pos = real ? position(a, b, j, (int64_t)__ldg(a.pool.lens + b) + j) : -1;
        float x[8] = {};
        if (real && (pos >= 0 || !a.rot))   // rows that are not there, or have no angle: 0
            load8(static_cast<const T *>(a.q) + b * a.qs[0] + j * a.qs[1] + h * a.qs[2] + d0, x);
        rotate8(x, a, d0, pos, real && a.rot && pos >= 0);
        if (on) store8(static_cast<T *>(a.q_out) + row * D + d0, x);
        return;
    }
    __shared__ float red[4][2][D];
    const int c = (int)(blockIdx.x % chunks);
    const int h = (int)(blockIdx.x / chunks % a.pool.Hkv);
    const int b = (int)(blockIdx.x / chunks / a.pool.Hkv);
    const int64_t len = __ldg(a.pool.lens + b);
    if (len < 0) {
        if (threadIdx.x == 0) kv4_report(a.pool.err);
        return;
    }
    const int64_t end = len + new_tokens(a, b);
    const int64_t c0 = ((len >> chunk_shift) + c) << chunk_shift;   // first slot of the chunk
    if (c0 >= end) return;
    const int chunk = 1 << chunk_shift;
    const int ps = a.pool.page_shift;
    const bool is_v = (lane / LPR) & 1;
    const int tsub = lane / (2 * LPR);
    float lo[8], hi[8];   // per-d extremes of the K rows that this lane has seen
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
    for (int s0 = warp * KV4_BLOCK; s0 < chunk; s0 += 4 * KV4_BLOCK) {
        const int64_t slot0 = c0 + s0;
        if (slot0 >= end || slot0 + KV4_BLOCK <= len) continue;
        const int id = kv4_page(a.pool, b, slot0 >> ps);
        if (id < 0) continue;
        uint8_t *blk = kv4_block<D>(a.pool, id, h, (int)((slot0 & ((1 << ps) - 1)) >> 4));
        const int t_lo = len > slot0 ? (int)(len - slot0) : 0;
        const int t_hi = end - slot0 < KV4_BLOCK ? (int)(end - slot0) : KV4_BLOCK;
        for (int t0 = t_lo; t0 < t_hi; t0 += TPI) {
            const int t = t0 + tsub;
            const int j = (int)(slot0 + t - len);
            bool on = t < t_hi;
            const int64_t pos = on ? position(a, b, j, slot0 + t) : -1;
            if (a.rot) on = on && pos >= 0;
            float x[8] = {};
            if (on) {
                const int64_t *st = is_v ? a.vs : a.ks;
                load8(static_cast<const T *>(is_v ? a.v : a.k) + b * st[0] + j * st[1] + h * st[2] + d0, x);
            }
            rotate8(x, a, d0, pos, on && a.rot && !is_v);
            int code[8];
            __half s, m;
            quantise8(x, code, s, m);
            if (!on) continue;
            const int gr = sub >> 2, q4 = sub & 3;
            if (!is_v) {
                uint32_t w = 0;
#pragma unroll
                for (int o = 0; o < 8; ++o) w |= (uint32_t)code[o] << (4 * ((o >> 1) + 4 * (o & 1)));
                *reinterpret_cast<uint32_t *>(blk + t * (D / 2) + (q4 * NG + gr) * 4) = w;
                if (q4 == 0)
                    *reinterpret_cast<__half2 *>(blk + Kv4<D>::K_META + (t * NG + gr) * 4) = __halves2half2(s, m);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool fin = isfinite(x[i]);
                    lo[i] = fminf(lo[i], fin ? x[i] : -INFINITY);
                    hi[i] = fmaxf(hi[i], fin ? x[i] : INFINITY);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w = code[4 * e] | code[4 * e + 1] << 4 | code[4 * e + 2] << 8 | code[4 * e + 3] << 12;
                    *reinterpret_cast<uint16_t *>(blk + v_code_at<D>(t, gr, 2 * q4 + e)) = (uint16_t)w;
                }
                if (q4 == 0) {
                    uint8_t *p = blk + v_meta_at<D>(t, gr);
                    *reinterpret_cast<__half *>(p) = s;
                    *reinterpret_cast<__half *>(p + 4) = m;
                }
            }
        }
        // __syncwarp is implied by the warp-wide shuffles of the next block
    }
    if (!a.summary) return;
    // extremes over the warp's token slots (D = 64: two per pass), then over the
    // warps that share a page
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (TPI == 2) {
            lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], 16));
            hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], 16));
        }
        if (!is_v && tsub == 0) red[warp][0][d0 + i] = lo[i], red[warp][1][d0 + i] = hi[i];
    }
    __syncthreads();
    const int share = (1 << ps) >= 64 ? 4 : (1 << ps) / KV4_BLOCK;   // warps that share a page
    for (int x = threadIdx.x; x < (4 / share) * 2 * D; x += 128) {
        const int p = x / (2 * D), mx = x / D & 1, d = x % D;
        const int64_t p0 = c0 + ((int64_t)p << ps);   // first slot of the page
        if (p0 >= end || p0 + (1 << ps) <= len) continue;
        float r = red[p * share][mx][d];
        for (int w = 1; w < share; ++w) r = mx ? fmaxf(r, red[p * share + w][mx][d]) : fminf(r, red[p * share + w][mx][d]);
        const int id = kv4_page(a.pool, b, p0 >> ps);
        if (id < 0) continue;
        __nv_bfloat16 *to = a.summary + (((int64_t)id * a.pool.Hkv + h) * 2 + mx) * D + d;
        if (p0 < len) {
            const float old = __bfloat162float(*to);
            r = mx ? fmaxf(r, old) : fminf(r, old);
        }
        *to = __float2bfloat16_rn(r);
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

__device__ __forceinline__ void store4(float *p, const float (&x)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&x)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}

template <int D, typename T>
__global__ void __launch_bounds__(128) kv4_gather_kernel(Kv4GatherArgs a, int blocks, int64_t warps)
{
    constexpr int NG = Kv4<D>::NG;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (wid >= warps) return;
    // heads next to each other: their rows are neighbours in k and v
    const int h = (int)(wid % a.pool.Hkv);
    const int x = (int)(wid / a.pool.Hkv % blocks);
    const int b = (int)(wid / a.pool.Hkv / blocks);
    const int len = kv4_len(a.pool, b);
    int64_t first = a.start ? (int64_t)__ldg(a.start + b) : 0;
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
    const int64_t q_rows = a.q ? (int64_t)a.B * a.n * a.Hq : 0;
    const int rpb = 128 / (D / 8);
    const int64_t blocks = kv_blocks + (q_rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffffLL) return CP_EUNSUPPORTED;
#define CP_KV4_APPEND(D_, T_) \
    kv4_append_kernel<D_, T_><<<(unsigned)blocks, 128, 0, st>>>(a, chunk_shift, (int)chunks, kv_blocks)
    if (D == 64) {
        if (dtype == CP_BF16) CP_KV4_APPEND(64, __nv_bfloat16);
        else CP_KV4_APPEND(64, float);
    } else {
        if (dtype == CP_BF16) CP_KV4_APPEND(128, __nv_bfloat16);
        else CP_KV4_APPEND(128, float);
    }
#undef CP_KV4_APPEND
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

int launch_kv4_gather(const Kv4GatherArgs &a, int D, int dtype, cudaStream_t st)
{
    // an unaligned start reaches one block more
    const int64_t blocks = ((int64_t)a.count + KV4_BLOCK - 2) / KV4_BLOCK + 1;
    const int64_t warps = blocks * a.pool.Hkv * a.B;
    const int64_t grid = (warps + 3) / 4;
    if (grid > 0x7fffffffLL) return CP_EUNSUPPORTED;
#define CP_KV4_GATHER(D_, T_) \
    kv4_gather_kernel<D_, T_><<<(unsigned)grid, 128, 0, st>>>(a, (int)blocks, warps)
    if (D == 64) {
        if (dtype == CP_BF16) CP_KV4_GATHER(64, __nv_bfloat16);
        else CP_KV4_GATHER(64, float);
    } else {
        if (dtype == CP_BF16) CP_KV4_GATHER(128, __nv_bfloat16);
        else CP_KV4_GATHER(128, float);
    }
#undef CP_KV4_GATHER
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace cp
