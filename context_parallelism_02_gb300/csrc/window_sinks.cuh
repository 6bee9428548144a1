// window_sinks.cuh -- the sinks' gradients of a windowed attention.  A sink is seen by
// every later row, too long a walk for one block, so the rows behind its window are
// cut into pieces (SinkPlan) whose partial dK and dV lie in the workspace and are
// added up here.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cp_common.cuh"

namespace cp {

// Tiles of the fp32 kernels: ROWS rows stay with a block (queries, or keys in dK / dV) while
// tiles of COLS pass by.  dK / dV gives the heads of a group to a cluster of blocks.
constexpr int WINDOW_F32_ROWS = 32, WINDOW_F32_COLS = 64;
CP_HD int window_f32_cluster(int grp)   // the largest divisor of the group up to 8
{
    int c = grp < 8 ? grp : 8;
    while (grp % c) --c;
    return c;
}
CP_HD SinkPlan window_f32_plan(const Window &w, int Sq, int grp, int64_t heads)
{
    return sink_plan<WINDOW_F32_ROWS, WINDOW_F32_COLS>(w, Sq, Sq + w.off, grp / window_f32_cluster(grp), heads);
}

// Partial gradients, fp32, [B][Hkv][1 + pieces][2 (dK, dV)][sinks][D]: slot 0 from the
// window unit of the key's tile, the others from the pieces.
CP_HD int64_t window_part_rows(const Window &w, const SinkPlan &s) { return (int64_t)(1 + s.pieces) * 2 * w.sinks; }

#if defined(__CUDACC__)

__device__ __forceinline__ void put_element(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put_element(float *p, float x) { *p = x; }

// One block per (batch, kv head, sink): eight runs of slots side by side, each in order,
// so the sums repeat bit for bit.
template <int D, typename Out>
__global__ void __launch_bounds__(8 * 64)
    window_sinks_kernel(const float *__restrict__ parts, const Window w, const SinkPlan sp, int Hkv, int Sk,
                        Out *__restrict__ dk, Out *__restrict__ dv)
{
    constexpr int E = 2 * D / 64;   // of dK's and dV's 2 D elements, per thread
    __shared__ float sum[8][2 * D];
    const int key = (int)(blockIdx.x % (unsigned)w.sinks);
    const unsigned bh = blockIdx.x / (unsigned)w.sinks;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    const float *part = parts + (int64_t)bh * window_part_rows(w, sp) * D;
    float s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = 0.f;
    const int slots = 1 + sp.pieces, run = (slots + 7) / 8;
#pragma unroll 4
    for (int i = y * run; i < min((y + 1) * run, slots); ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int el = x + 64 * e, which = el / D;
            s[e] += part[(((int64_t)i * 2 + which) * w.sinks + key) * D + el % D];
        }
#pragma unroll
    for (int e = 0; e < E; ++e) sum[y][x + 64 * e] = s[e];
    __syncthreads();
    if (threadIdx.x >= 2 * D) return;
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) r += sum[i][threadIdx.x];
    const unsigned b = bh / (unsigned)Hkv, h = bh % (unsigned)Hkv;
    const int which = threadIdx.x / D;
    put_element((which ? dv : dk) + (((int64_t)b * Sk + key) * Hkv + h) * D + threadIdx.x % D, r);
}

template <int D, typename Out>
int launch_window_sinks(const float *parts, const Window &w, const SinkPlan &sp, int B, int Hkv, int Sk, Out *dk,
                        Out *dv, cudaStream_t st)
{
    if (!sp.pieces) return CP_OK;
    const int64_t blocks = (int64_t)B * Hkv * w.sinks;
    if (blocks > 0x7fffffffLL) return CP_EUNSUPPORTED;
    window_sinks_kernel<D, Out><<<(unsigned)blocks, 512, 0, st>>>(parts, w, sp, Hkv, Sk, dk, dv);
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

#endif

}  // namespace cp
