// window_fix.cuh -- windowed attention's rows that values outside their reach have spoilt.
//
// A tile's products take every key of the tile for every row, with weight 0 where the mask
// hides it; but 0 times a NaN or an infinity is NaN, and what lies outside a row's window
// may hold anything (the padding of a batch, rows that were never written).  So a result
// that is not finite is noted, and when the block has done all its units its warps compute
// the noted rows again, over the visible keys alone.  Results that are finite have met no
// such value, so a call without any pays a sum a row.  Only elements that are not finite are
// replaced, and a row is left as soon as none of them can become finite any more: tensors
// that are NaN throughout cost a key a row and not all of them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cp_common.cuh"
#include "tc_helpers.cuh"

namespace cp {

#if defined(__CUDACC__)

// Notes of a block: (unit of the block, warp) pairs; past CAP all of them count as noted.
struct FixList {
    static constexpr int CAP = 56;
    int count, entry[CAP];
    __device__ __forceinline__ void note(int unit, int warp)
    {
        const int at = atomicAdd(&count, 1);
        if (at < CAP) entry[at] = unit * 8 + warp;
    }
};

// What the recomputation reads; Sq rows, Sk keys.
struct FixArgs {
    const __nv_bfloat16 *q, *k, *v, *out, *dout;
    const float *lse, *delta;
    int Sq, Sk, Hq, Hkv;
    float scale;
    Window win;
};

namespace fix {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

// The lane's D / 32 elements of a row.
template <int D>
struct Piece {
    float x[D / 32];
};
template <int D>
__device__ __forceinline__ Piece<D> load(const __nv_bfloat16 *row, int lane)
{
    Piece<D> p;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const float2 f = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(row)[lane + 32 * i]);
        p.x[2 * i] = f.x;
        p.x[2 * i + 1] = f.y;
    }
    return p;
}
template <int D>
__device__ __forceinline__ void store(__nv_bfloat16 *row, const Piece<D> &p, int lane)
{
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        reinterpret_cast<uint32_t *>(row)[lane + 32 * i] = tc::pack_bf16(p.x[2 * i], p.x[2 * i + 1]);
}
template <int D>
__device__ __forceinline__ float dot(const Piece<D> &a, const Piece<D> &b)
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(a.x[i], b.x[i], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
template <int D>
__device__ __forceinline__ bool finite(const Piece<D> &p)
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(p.x[i], 0.f, s);
    return __all_sync(0xffffffffu, s == s);
}

// Whether no element that was not finite can become so: the sums of all of them are not.
template <int D>
__device__ __forceinline__ bool lost(const Piece<D> &was, const Piece<D> &acc)
{
    bool all = true;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) all = all && (was.x[e] * 0.f == 0.f || !(acc.x[e] * 0.f == 0.f));
    return __all_sync(0xffffffffu, all);
}
// What was finite stays, the rest is taken from acc, times f.
template <int D>
__device__ __forceinline__ Piece<D> mended(const Piece<D> &was, const Piece<D> &acc, float f)
{
    Piece<D> p;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) p.x[e] = was.x[e] * 0.f == 0.f ? was.x[e] : acc.x[e] * f;
    return p;
}

// f(key) for the keys that the row at position p sees, until it returns true.
template <typename F>
__device__ __forceinline__ void each_key(const Window &w, int p, F f)
{
    const int lo = p - w.window + 1 > 0 ? p - w.window + 1 : 0;
    for (int j = 0; j < w.sinks && j < lo; ++j)
        if (f(j)) return;
    for (int j = lo; j <= p; ++j)
        if (f(j)) return;
}

// Output row i of (b, h).
template <int D>
__device__ __noinline__ void out_row(const FixArgs &a, int b, int h, int i, __nv_bfloat16 *out)
{
    const int lane = threadIdx.x & 31, kvh = h / (a.Hq / a.Hkv);
    __nv_bfloat16 *row = out + (((int64_t)b * a.Sq + i) * a.Hq + h) * D;
    const Piece<D> was = load<D>(row, lane);
    if (finite(was)) return;
    const Piece<D> q = load<D>(a.q + (((int64_t)b * a.Sq + i) * a.Hq + h) * D, lane);
    const float z = a.lse[((int64_t)b * a.Hq + h) * a.Sq + i] * LOG2E, sl2 = a.scale * LOG2E;
    Piece<D> acc{};
    each_key(a.win, i + a.win.off, [&](int j) {
        const int64_t at = (((int64_t)b * a.Sk + j) * a.Hkv + kvh) * D;
        const float p = tc::ex2(fmaf(dot(q, load<D>(a.k + at, lane)), sl2, -z));
        const Piece<D> v = load<D>(a.v + at, lane);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc.x[e] = fmaf(p, v.x[e], acc.x[e]);
        return lost(was, acc);
    });
    store(row, mended(was, acc, 1.f), lane);
}

// dQ row i of (b, h).
template <int D>
__device__ __noinline__ void dq_row(const FixArgs &a, int b, int h, int i, __nv_bfloat16 *dq)
{
    const int lane = threadIdx.x & 31, kvh = h / (a.Hq / a.Hkv);
    const int64_t at_q = (((int64_t)b * a.Sq + i) * a.Hq + h) * D;
    const Piece<D> was = load<D>(dq + at_q, lane);
    if (finite(was)) return;
    const Piece<D> q = load<D>(a.q + at_q, lane), g = load<D>(a.dout + at_q, lane);
    const int64_t stat = ((int64_t)b * a.Hq + h) * a.Sq + i;
    const float z = a.lse[stat] * LOG2E, dl = a.delta[stat], sl2 = a.scale * LOG2E;
    Piece<D> acc{};
    each_key(a.win, i + a.win.off, [&](int j) {
        const int64_t at = (((int64_t)b * a.Sk + j) * a.Hkv + kvh) * D;
        const Piece<D> k = load<D>(a.k + at, lane);
        const float ds = tc::ex2(fmaf(dot(q, k), sl2, -z)) * (dot(g, load<D>(a.v + at, lane)) - dl);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc.x[e] = fmaf(ds, k.x[e], acc.x[e]);
        return lost(was, acc);
    });
    store(dq + at_q, mended(was, acc, a.scale), lane);
}

// dK or dV of key j of (b, kv head) over rows [i0, i1) of head h, added to acc; true: lost.
template <int D>
__device__ __noinline__ bool key_rows(const FixArgs &a, int b, int h, int j, int i0, int i1, bool want_k, const Piece<D> &was,
                                      Piece<D> &acc)
{
    const int lane = threadIdx.x & 31, kvh = h / (a.Hq / a.Hkv);
    const int64_t at = (((int64_t)b * a.Sk + j) * a.Hkv + kvh) * D;
    const Piece<D> k = load<D>(a.k + at, lane), v = load<D>(a.v + at, lane);
    const float sl2 = a.scale * LOG2E;
    for (int i = i0; i < i1; ++i) {
        const int64_t at_q = (((int64_t)b * a.Sq + i) * a.Hq + h) * D, stat = ((int64_t)b * a.Hq + h) * a.Sq + i;
        const Piece<D> q = load<D>(a.q + at_q, lane), g = load<D>(a.dout + at_q, lane);
        const float p = tc::ex2(fmaf(dot(q, k), sl2, -a.lse[stat] * LOG2E));
        const float f = want_k ? p * (dot(g, v) - a.delta[stat]) * a.scale : p;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc.x[e] = fmaf(f, want_k ? q.x[e] : g.x[e], acc.x[e]);
        if (lost(was, acc)) return true;
    }
    return false;
}

}  // namespace fix

#endif

}  // namespace cp
