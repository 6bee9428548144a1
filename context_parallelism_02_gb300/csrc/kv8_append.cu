// kv8_append.cu -- new tokens into the paged 8-bit cache, and cached tokens back as rows.
//
// Append, per block of 16 tokens, kv head and K or V: the block's scale is that of the
// largest magnitude among its tokens, so one warp takes all of a block's new rows:
//   amax over them, e = exponent of the scale (kv8_scale_of), scale = max(old, 2^e),
//   code = e4m3(x / scale);  where the scale grew, the older codes are rounded to it.
// x / scale is exact, so a code is x rounded once.  Gather: value = code scale, exact in
// fp32 and in bf16 (e4m3's four bits times a power of two).
// Both move bytes: 3 D a row and K or V in bf16, and are bounded by HBM: 32768 tokens of 8
// heads, D = 128, 36 and 31 us each alone, 65 one behind the other (6.2 TB/s); single tokens
// by two chains of loads, 16 sequences 4.3 us for both.
#include "kernels.h"
#include "kv8.cuh"
#include "tc_helpers.cuh"

namespace cp {

namespace {

constexpr int WARPS = 8;

// How a warp lies over 16 rows of D elements of T: 16 bytes a lane, ROWS rows an access.
template <int D, typename T>
struct Lay {
    static constexpr int EPL = 16 / (int)sizeof(T);   // elements of a lane's access
    static constexpr int LANES = D / EPL;             // lanes of a row
    static constexpr int ROWS = 32 / LANES;
    static constexpr int N = 16 / ROWS;               // accesses
};

// The units of a launch: (batch, block, head, K or V), the last fastest, so that the warps of
// a moment read neighbouring rows.
struct Units {
    FastDiv by_heads, by_blocks;
    int n;
    __device__ __forceinline__ void decode(int unit, int &b, int &t, int &h, int &which) const
    {
        which = unit & 1;
        const unsigned x = (unsigned)unit >> 1, y = by_heads.div(x);
        h = (int)(x - y * by_heads.d);
        const unsigned z = by_blocks.div(y);
        t = (int)(y - z * by_blocks.d);
        b = (int)z;
    }
};

// The magnitudes' bits of the elements of 16 bytes: the largest, as fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const uint4 &x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) top = max(top, w[i] & 0x7fffffffu);
        else top = max(top, max((w[i] & 0x7fffu) << 16, w[i] & 0x7fff0000u));
    }
    return top;
}
// The same over the finite ones.
template <typename T>
__device__ __forceinline__ uint32_t top_finite(const uint4 &x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = sizeof(T) == 4 ? w[i] & 0x7fffffffu : (w[i] & 0x7fffu) << 16, b = w[i] & 0x7fff0000u;
        if (a < 0x7f800000u) top = max(top, a);
        if (sizeof(T) == 2 && b < 0x7f800000u) top = max(top, b);
    }
    return top;
}

template <typename T>
__device__ __forceinline__ float element(const uint4 &x, int i)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

// x / scale as codes; `odd`: some element is not finite, and infinities become NaN.
template <typename T>
__device__ __forceinline__ void encode(const uint4 &x, float inv, bool odd, uint32_t (&code)[Lay<64, T>::EPL / 4])
{
#pragma unroll
    for (int i = 0; i < Lay<64, T>::EPL / 4; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = element<T>(x, 4 * i + e);
            v[e] = f * inv;
            if (odd) v[e] = fmaf(f, 0.f, v[e]);
        }
        code[i] = kv8_codes4(v[0], v[1], v[2], v[3]);
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(WARPS * 32, sizeof(T) == 2 ? 4 : 2) kv8_append_kernel(Kv8AppendArgs a, Units units)
{
    using L = Lay<D, T>;
    const int lane = threadIdx.x & 31;
    kv4_begin();
    const int64_t unit = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (unit >= units.n) return;
    int b, t, h, which;
    units.decode((int)unit, b, t, h, which);
    const int64_t len = kv4_len(a.pool, b);
    const int n = a.n_new ? max(0, min(a.n_new[b], a.n)) : a.n;
    const int64_t slot0 = (len / KV8_BLOCK + t) * KV8_BLOCK;    // the block's first slot
    if (n == 0 || slot0 >= len + n) return;                     // (without new tokens: its pages may be gone)
    const int lo = slot0 < len ? (int)(len - slot0) : 0;        // rows [lo, hi) of the block are new
    const int hi = (int)(len + n - slot0 < KV8_BLOCK ? len + n - slot0 : KV8_BLOCK);
    const int64_t *st = which ? a.vs : a.ks;
    const T *src = static_cast<const T *>(which ? a.v : a.k) + b * st[0] + h * st[2] + lane % L::LANES * L::EPL;
    const int j0 = (int)(slot0 - len);                          // new token of row 0 (negative: an older one)
    const int r0 = lane / L::LANES;
    uint4 x[L::N];                                              // on their way while the page is looked up
#pragma unroll
    for (int i = 0; i < L::N; ++i) {
        const int r = r0 + i * L::ROWS;
        x[i] = r >= lo && r < hi ? *reinterpret_cast<const uint4 *>(src + (int64_t)(j0 + r) * st[1]) : make_uint4(0, 0, 0, 0);
    }
    const int id = kv4_page(a.pool, b, slot0 >> a.pool.page_shift);
    if (id < 0) return;
    const int at = (int)(slot0 & ((1 << a.pool.page_shift) - 1));
    float *sp = kv8_scale(a.pool, id, h, which, at);
    const float held = lo > 0 ? *sp : 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < L::N; ++i) top = max(top, top_bits<T>(x[i]));
    top = __reduce_max_sync(0xffffffffu, top);
    const bool odd = top >= 0x7f800000u;
    if (odd) {
        top = 0;
#pragma unroll
        for (int i = 0; i < L::N; ++i) top = max(top, top_finite<T>(x[i]));
        top = __reduce_max_sync(0xffffffffu, top);
    }
    const float made = kv8_scale_of(top), scale = lo > 0 ? fmaxf(held, made) : made, inv = 1.f / scale;
    uint8_t *row = kv8_row<D>(a.pool, id, h, which, at) + lane % L::LANES * L::EPL;
#pragma unroll
    for (int i = 0; i < L::N; ++i) {
        const int r = r0 + i * L::ROWS;
        if (r < lo || r >= hi) continue;
        uint32_t code[L::EPL / 4];
        encode<T>(x[i], inv, odd, code);
        if (sizeof(T) == 2) *reinterpret_cast<uint2 *>(row + r * D) = make_uint2(code[0], code[L::EPL / 4 - 1]);
        else *reinterpret_cast<uint32_t *>(row + r * D) = code[0];
    }
    if (lo > 0 && scale > held) {   // the older tokens' codes, rounded to the block's new scale
        uint32_t *old = reinterpret_cast<uint32_t *>(kv8_row<D>(a.pool, id, h, which, at));
        const float f = held / scale;
        for (int i = lane; i < lo * (D / 4); i += 32) old[i] = kv8_shrink(old[i], f);
    }
    if (lane == 0 && (lo == 0 || scale > held)) *sp = scale;
}

// 16 rows of one head: 8 codes a lane, so that reads and writes cover whole rows.
template <int D, bool BF16>
__global__ void __launch_bounds__(WARPS * 32) kv8_gather_kernel(Kv8GatherArgs a, Units units)
{
    constexpr int LANES = D / 8, ROWS = 32 / LANES, N = 16 / ROWS;
    const int lane = threadIdx.x & 31;
    kv4_begin();
    const int64_t unit = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (unit >= units.n) return;
    int b, t, h, which;
    units.decode((int)unit, b, t, h, which);
    const int64_t len = kv4_len(a.pool, b), start = a.start ? a.start[b] : 0;
    // lane r < 16: where row r comes from
    const uint8_t *src = nullptr;
    float scale = 0.f;
    {
        const int j = t * 16 + lane;
        const int64_t slot = start + j;
        if (lane < 16 && j < a.count && slot < len) {
            if (slot < 0) {
                kv4_report(a.pool.err);
            } else {
                const int id = kv4_page(a.pool, b, slot >> a.pool.page_shift);
                const int at = (int)(slot & ((1 << a.pool.page_shift) - 1));
                if (id >= 0) {
                    src = kv8_row<D>(a.pool, id, h, which, at);
                    scale = *kv8_scale(a.pool, id, h, which, at);
                }
            }
        }
    }
    uint2 x[N];
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = lane / LANES + i * ROWS;
        const uint8_t *p = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), r));
        x[i] = p ? *reinterpret_cast<const uint2 *>(p + lane % LANES * 8) : make_uint2(0, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __shfl_sync(0xffffffffu, scale, lane / LANES + i * ROWS);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = t * 16 + lane / LANES + i * ROWS;
        if (j >= a.count) continue;
        const int64_t at = (((int64_t)b * a.count + j) * a.pool.Hkv + h) * D + lane % LANES * 8;
        float4 u = kv8_floats(x[i].x), v = kv8_floats(x[i].y);
        u.x *= f[i], u.y *= f[i], u.z *= f[i], u.w *= f[i];
        v.x *= f[i], v.y *= f[i], v.z *= f[i], v.w *= f[i];
        if (BF16) {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(which ? a.v : a.k) + at) =
                make_uint4(tc::pack_bf16(u.x, u.y), tc::pack_bf16(u.z, u.w), tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
        } else {
            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(which ? a.v : a.k) + at);
            dst[0] = u;
            dst[1] = v;
        }
    }
}

template <typename A>
int launch_units(void (*kernel)(A, Units), const A &a, int64_t blocks, cudaStream_t st)
{
    const __int128 n = (__int128)a.B * blocks * a.pool.Hkv * 2;
    if (n > 0x7fffffff) return CP_EUNSUPPORTED;
    const Units units{fast_div((uint32_t)a.pool.Hkv), fast_div((uint32_t)blocks), (int)n};
    return kv4_launch(kernel, (unsigned)((n + WARPS - 1) / WARPS), WARPS * 32, 0, st, a, units) == cudaSuccess ? CP_OK : CP_ECUDA;
}

}  // namespace

int launch_kv8_append(const Kv8AppendArgs &a, int D, int dtype, cudaStream_t st)
{
    // n tokens behind any slot touch at most this many blocks
    const int64_t blocks = ((int64_t)a.n + KV8_BLOCK - 2) / KV8_BLOCK + 1;
    if (dtype == CP_BF16)
        return D == 64 ? launch_units(kv8_append_kernel<64, __nv_bfloat16>, a, blocks, st)
                       : launch_units(kv8_append_kernel<128, __nv_bfloat16>, a, blocks, st);
    return D == 64 ? launch_units(kv8_append_kernel<64, float>, a, blocks, st)
                   : launch_units(kv8_append_kernel<128, float>, a, blocks, st);
}

int launch_kv8_gather(const Kv8GatherArgs &a, int D, int dtype, cudaStream_t st)
{
    const int64_t blocks = ((int64_t)a.count + 15) / 16;
    if (dtype == CP_BF16)
        return D == 64 ? launch_units(kv8_gather_kernel<64, true>, a, blocks, st)
                       : launch_units(kv8_gather_kernel<128, true>, a, blocks, st);
    return D == 64 ? launch_units(kv8_gather_kernel<64, false>, a, blocks, st)
                   : launch_units(kv8_gather_kernel<128, false>, a, blocks, st);
}

}  // namespace cp
