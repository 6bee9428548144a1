// kv8.cuh -- the paged 8-bit key/value cache: its format and the arguments of its kernels.
//
// The pool is [n_pages][Hkv][2 (K, V)][page][D] bytes, codes in e4m3 (8 bits: sign, four
// bits of exponent, three of mantissa, +-448 at most, no infinities), rows as they are,
// so that a row is one run of D bytes for whoever reads, writes or moves it.  The scales
// are [n_pages][Hkv][2][page / 16] fp32: one for the 16 tokens of a block, a power of two
// 2^e, e the smallest in [-40, 60] with amax <= 448 2^e.  A value is code 2^e.
// Powers of two make scaling exact: a code is its value rounded once, and stays so when
// its block's scale grows, unless it falls below e4m3's normal range.
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace cp {

constexpr int KV8_BLOCK = 16;              // tokens that share a scale
constexpr int KV8_E_MIN = -40, KV8_E_MAX = 60;

struct Kv8Pool : Kv4Pool {                 // data: the codes
    float *scales;
};

#if defined(__CUDACC__)

// Number of (page, kv head, K or V) in the pool's order.
__device__ __forceinline__ int64_t kv8_plane(const Kv8Pool &c, int id, int h, int which)
{
    return ((int64_t)id * c.Hkv + h) * 2 + which;
}
// The row of slot `at` of a page, and the scale of its block.
template <int D>
__device__ __forceinline__ uint8_t *kv8_row(const Kv8Pool &c, int id, int h, int which, int at)
{
    return c.data + ((kv8_plane(c, id, h, which) << c.page_shift) + at) * D;
}
__device__ __forceinline__ float *kv8_scale(const Kv8Pool &c, int id, int h, int which, int at)
{
    return c.scales + (kv8_plane(c, id, h, which) << (c.page_shift - 4)) + (at >> 4);
}

// The scale for a largest magnitude of the given fp32 bits (finite): with amax = m 2^x,
// m in [1, 2), 448 = 1.75 2^8 leaves e = x - 8, one more where m > 1.75.
__device__ __forceinline__ float kv8_scale_of(uint32_t amax)
{
    int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < KV8_E_MIN ? KV8_E_MIN : e > KV8_E_MAX ? KV8_E_MAX : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two values to two codes (nearest even, held within +-448; NaN stays NaN), the first low.
__device__ __forceinline__ uint32_t kv8_codes2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// Four values to a word of codes.
__device__ __forceinline__ uint32_t kv8_codes4(float a, float b, float c, float d)
{
    return kv8_codes2(a, b) | kv8_codes2(c, d) << 16;
}
// Two codes to two fp16 (exact).
__device__ __forceinline__ uint32_t kv8_halves(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// Four codes to fp32.
__device__ __forceinline__ float4 kv8_floats(uint32_t four)
{
    const uint32_t lo = kv8_halves(four & 0xffffu), hi = kv8_halves(four >> 16);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
}
// Codes whose block's scale grows by 1 / f (f a power of two below 1).
__device__ __forceinline__ uint32_t kv8_shrink(uint32_t four, float f)
{
    const float4 v = kv8_floats(four);
    return kv8_codes4(v.x * f, v.y * f, v.z * f, v.w * f);
}

#endif

struct Kv8AppendArgs {
    Kv8Pool pool;                // lens: tokens before the append
    const void *k, *v;
    const int32_t *n_new;        // [B] or null
    int64_t ks[3], vs[3];        // element strides of batch, token, head
    int B, n;
};
int launch_kv8_append(const Kv8AppendArgs &a, int D, int dtype, cudaStream_t st);

struct Kv8GatherArgs {
    Kv8Pool pool;
    const int32_t *start;        // [B] or null (0)
    void *k, *v;                 // [B][count][Hkv][D]
    int B, count;
};
int launch_kv8_gather(const Kv8GatherArgs &a, int D, int dtype, cudaStream_t st);

struct Kv8AttnArgs {
    Kv8Pool pool;
    Kv4Rows rows;
    const __nv_bfloat16 *q;      // [B][n][Hq][D]
    void *out;                   // [B][n][Hq][D]
    float *lse;                  // [B][Hq][n]
    float *mass;                 // [B][Hkv][max_pages page] or null
    float *scores;               // [B][Hkv][max_pages page][n Hq / Hkv, to a multiple of 4], log2 units
    int window, sinks;           // window 0: none
    int out_f32;
    float scale;
    void *ws;
    uint64_t limit_ns, drain_ns;
};
size_t kv8_attn_workspace_bytes(int B, int n, int Hq, int Hkv, int D, int64_t slots, bool mass);
int launch_kv8_attn(const Kv8AttnArgs &a, int D, int64_t n_pages, cudaStream_t st);

struct Kv8EvictArgs {
    Kv8Pool pool;
    const float *mass;           // [B][Hkv][max_pages page]
    const int32_t *to;           // [B][max_to]
    int32_t *kept, *lens_to;     // [B][Hkv][budget], [B]
    float *mass_to;              // [B][Hkv][max_to page] or null
    int B, max_to, budget, first, last;
};
int launch_kv8_evict(const Kv8EvictArgs &a, int D, cudaStream_t st);

}  // namespace cp
