// window_f32.cu -- windowed attention with sinks on fp32 tensors, forward and backward,
// on the CUDA cores in fp32 arithmetic (bounded by the FMA pipe: no tensor-core kind
// holds fp32's 24 bits).
//
// Tiles of 32 rows by 64 columns, 128 threads as 8 x 16, each with a 4 x 4 part of the
// scores (rows ty + 8 i, columns tx + 16 j) and of the 32 x D products 4 rows by D / 16
// columns (4 tx + 64 j).  Per four elements of the inner axis a thread reads 8 x 16 bytes
// of shared memory for 64 FMAs, which go in pairs.  Small blocks, several to an SM, cover
// each other's loads and leave less behind the mask than 64 x 64 tiles of 256 threads.
// A step of 2 x 1001 rows, 6 heads on 2, D = 64, window 200, 5 sinks takes 137 us; 162 with
// single FMAs and a tile for the sinks alone, 318 with the large tiles (212 with the small
// ones at the same stage).  The walks are those of the bf16 kernels: WinIter for the
// query-stationary kernels, WinQIter and the sinks' pieces for dK and dV, whose heads of a
// group go to the blocks of a cluster and are added up in order through distributed shared
// memory; every output element is written once.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "cp_common.cuh"
#include "kernels.h"
#include "tc_helpers.cuh"
#include "window_sinks.cuh"

namespace cp {

namespace {

namespace cg = cooperative_groups;

constexpr int R = WINDOW_F32_ROWS, T = WINDOW_F32_COLS;
constexpr int THREADS = 128;
constexpr int PS = T + 4;             // row stride of an R x T tile in shared memory
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994530942f;

template <int D>
struct Rows {
    static constexpr int STRIDE = D + 4;        // a warp's 8 rows of 16 bytes fall on 32 banks
    static constexpr int FEW = R * STRIDE, FLOATS = T * STRIDE;
};

struct Args {
    const float *q, *k, *v, *out, *dout, *lse;
    float *delta, *part;
    int B, Hq, Hkv, Sq, Sk;
    float scale;
    Window win;
    SinkPlan sp;
};

// n rows of x [B][S][H][D] (head h, from row r0; the first pk of them from row 0) into COUNT rows
// of shared memory, the rest 0.  Returns NaN if one of the thread's elements is not finite, else 0.
template <int D, int COUNT>
__device__ __forceinline__ float load_rows(float *dst, const float *x, int64_t b, int S, int H, int h, int r0, int n,
                                           int pk = 0)
{
    float odd = 0.f;
#pragma unroll 8
    for (int i = threadIdx.x; i < COUNT * (D / 4); i += THREADS) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) v = *reinterpret_cast<const float4 *>(x + ((b * S + (r < pk ? r : r0 + r)) * H + h) * D + c * 4);
        *reinterpret_cast<float4 *>(dst + r * Rows<D>::STRIDE + c * 4) = v;
        odd = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, odd))));
    }
    return odd;
}

// acc[i][j] = A[ty + 8 i] . B[tx + 16 j]
template <int D>
__device__ __forceinline__ void dots(const float *A, const float *B, float (&acc)[4][4])
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float even[4][4], odd[4][4];   // sums over the even and the odd elements: pairs of FMAs
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) even[i][j] = odd[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4 *>(A + (ty + 8 * i) * Rows<D>::STRIDE + d);
            b[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * Rows<D>::STRIDE + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                tc::ffma2v(even[i][j], odd[i][j], a[i].x, a[i].y, b[j].x, b[j].y, even[i][j], odd[i][j]);
                tc::ffma2v(even[i][j], odd[i][j], a[i].z, a[i].w, b[j].z, b[j].w, even[i][j], odd[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = even[i][j] + odd[i][j];
}

// acc[i][4 j + e] += sum_k P[ty + 8 i][k] B[k][4 tx + 64 j + e].  `odd`: B holds values that are
// not finite, which a weight of 0 (what the mask hides) must not carry into the sums.
template <int D>
__device__ __forceinline__ void product(const float *P, const float *B, bool odd, float (&acc)[4][D / 16])
{
    if (odd) {
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 1
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = P[(ty + 8 * i) * PS + k];
                if (p == 0.f) continue;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(B + k * Rows<D>::STRIDE + 4 * tx + 64 * j);
                    acc[i][4 * j + 0] = fmaf(p, b.x, acc[i][4 * j + 0]);
                    acc[i][4 * j + 1] = fmaf(p, b.y, acc[i][4 * j + 1]);
                    acc[i][4 * j + 2] = fmaf(p, b.z, acc[i][4 * j + 2]);
                    acc[i][4 * j + 3] = fmaf(p, b.w, acc[i][4 * j + 3]);
                }
            }
        return;
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
    for (int k = 0; k < T; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(P + (ty + 8 * i) * PS + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const float4 b = *reinterpret_cast<const float4 *>(B + (k + kk) * Rows<D>::STRIDE + 4 * tx + 64 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                    float *o = &acc[i][4 * j];
                    tc::ffma2v(o[0], o[1], x, x, b.x, b.y, o[0], o[1]);
                    tc::ffma2v(o[2], o[3], x, x, b.z, b.w, o[2], o[3]);
                }
            }
    }
}

// What thread row i of the walk's current tile sees: columns [lo, hi) and [0, sc).
struct Seen {
    int lo, hi, sc;
    __device__ __forceinline__ Seen(const WinIter<T> &it, const Window &w, int p)
    {
        const int kl = it.len(), ks = it.start();
        hi = p - ks + 1 < kl ? p - ks + 1 : kl;
        lo = it.window_col(w, p);
        sc = it.sink_cols();
    }
    __device__ __forceinline__ bool at(int c) const { return c < hi && (c >= lo || c < sc); }
};

__device__ __forceinline__ float row_max(float x)   // over the 16 threads of a row
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The unit's query rows: heads fastest, so that the heads of a group share K and V in L2.
struct QUnit {
    int b, h, kvh, q0, rows;
    __device__ __forceinline__ QUnit(const Args &a)
    {
        unsigned u = blockIdx.x;
        h = (int)(u % (unsigned)a.Hq);
        u /= (unsigned)a.Hq;
        b = (int)(u % (unsigned)a.B);
        q0 = (int)(u / (unsigned)a.B) * R;
        kvh = h / (a.Hq / a.Hkv);
        rows = a.Sq - q0 < R ? a.Sq - q0 : R;
    }
};

// Rows of K or V for the walk's current tile; a packed one begins with the sinks.
template <int D>
__device__ __forceinline__ float load_keys(float *dst, const float *x, const Args &a, const QUnit &u, const WinIter<T> &it)
{
    return load_rows<D, T>(dst, x, u.b, a.Sk, a.Hkv, u.kvh, it.start(), it.len(), it.packed() ? it.pk : 0);
}

template <int D>
__global__ void __launch_bounds__(THREADS) window_f32_fwd_kernel(const Args a, float *__restrict__ out, float *__restrict__ lse)
{
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + Rows<D>::FEW, *V = K + Rows<D>::FLOATS, *P = V + Rows<D>::FLOATS;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const QUnit u(a);
    load_rows<D, R>(Q, a.q, u.b, a.Sq, a.Hq, u.h, u.q0, u.rows);
    const float sl2 = a.scale * LOG2E;
    float o[4][D / 16], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
    }
    const int p0 = u.q0 + a.win.off, p1 = p0 + u.rows - 1;
    WinIter<T> it;
    for (it.begin(a.win, p0, p1); it.valid(); it.next()) {
        __syncthreads();
        load_keys<D>(K, a.k, a, u, it);
        const float odd_v = load_keys<D>(V, a.v, a, u, it);
        const bool odd = __syncthreads_or(odd_v != odd_v);
        float x[4][4];
        dots<D>(Q, K, x);
        const bool full = it.full(a.win, p0, p1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Seen see(it, a.win, p0 + ty + 8 * i);
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = full || see.at(tx + 16 * j) ? x[i][j] * sl2 : -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
            const float mn = fmaxf(m[i], row_max(top)), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);   // 0 where nothing was seen before
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (a visible weight is never 0: product() skips those)
                const float w = exp2f(x[i][j] - base);
                x[i][j] = x[i][j] == -INFINITY ? 0.f : w == 0.f ? 1e-45f : w;
                sum += x[i][j];
                P[(ty + 8 * i) * PS + tx + 16 * j] = x[i][j];
            }
            l[i] = l[i] * f + row_sum(sum);
            m[i] = mn;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[i][j] *= f;
        }
        __syncthreads();
        product<D>(P, V, odd, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 8 * i;
        if (r >= u.rows) continue;
        const float inv = 1.f / l[i];           // a row sees itself; NaN where it sees a NaN
        float *row = out + (((int64_t)u.b * a.Sq + u.q0 + r) * a.Hq + u.h) * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            *reinterpret_cast<float4 *>(row + 4 * tx + 64 * j) =
                make_float4(o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv);
        // (a sum of 0: all its scores are -infinity, and -infinity would be the lse of an empty row)
        if (tx == 0)
            lse[((int64_t)u.b * a.Hq + u.h) * a.Sq + u.q0 + r] = l[i] == 0.f ? __int_as_float(0x7fffffff) : fmaf(m[i], LN2, logf(l[i]));
    }
}

// Delta = rowsum(dO * out), a warp a row.
template <int D>
__global__ void __launch_bounds__(THREADS) window_f32_delta_kernel(const Args a)
{
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.B * a.Sq * a.Hq, step = (int64_t)gridDim.x * (THREADS / 32);
    for (int64_t r = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); r < rows; r += step) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) s = fmaf(a.dout[r * D + lane + 32 * e], a.out[r * D + lane + 32 * e], s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int64_t bs = r / a.Hq, h = r % a.Hq, b = bs / a.Sq;
        if (lane == 0) a.delta[(b * a.Hq + h) * a.Sq + bs % a.Sq] = s;
    }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 3) window_f32_dq_kernel(const Args a, float *__restrict__ dq)
{
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *G = Q + Rows<D>::FEW, *K = G + Rows<D>::FEW, *V = K + Rows<D>::FLOATS, *P = V + Rows<D>::FLOATS;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const QUnit u(a);
    load_rows<D, R>(Q, a.q, u.b, a.Sq, a.Hq, u.h, u.q0, u.rows);
    load_rows<D, R>(G, a.dout, u.b, a.Sq, a.Hq, u.h, u.q0, u.rows);
    const float sl2 = a.scale * LOG2E;
    float acc[4][D / 16], lse2[4], delta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 8 * i;
        const int64_t at = ((int64_t)u.b * a.Hq + u.h) * a.Sq + u.q0 + r;
        lse2[i] = r < u.rows ? a.lse[at] * LOG2E : 0.f;
        delta[i] = r < u.rows ? a.delta[at] : 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
    }
    const int p0 = u.q0 + a.win.off, p1 = p0 + u.rows - 1;
    WinIter<T> it;
    for (it.begin(a.win, p0, p1); it.valid(); it.next()) {
        __syncthreads();
        const float odd_k = load_keys<D>(K, a.k, a, u, it);
        load_keys<D>(V, a.v, a, u, it);
        const bool odd = __syncthreads_or(odd_k != odd_k);
        float x[4][4], g[4][4];
        dots<D>(Q, K, x);
        dots<D>(G, V, g);
        const bool full = it.full(a.win, p0, p1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Seen see(it, a.win, p0 + ty + 8 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = full || see.at(tx + 16 * j);
                P[(ty + 8 * i) * PS + tx + 16 * j] = on ? exp2f(fmaf(x[i][j], sl2, -lse2[i])) * (g[i][j] - delta[i]) : 0.f;
            }
        }
        __syncthreads();
        product<D>(P, K, odd, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 8 * i;
        if (r >= u.rows) continue;
        float *row = dq + (((int64_t)u.b * a.Sq + u.q0 + r) * a.Hq + u.h) * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            *reinterpret_cast<float4 *>(row + 4 * tx + 64 * j) =
                make_float4(acc[i][4 * j] * a.scale, acc[i][4 * j + 1] * a.scale, acc[i][4 * j + 2] * a.scale,
                            acc[i][4 * j + 3] * a.scale);
    }
}

template <int D>
__global__ void __launch_bounds__(THREADS) window_f32_dkdv_kernel(const Args a, float *__restrict__ dk, float *__restrict__ dv)
{
    extern __shared__ __align__(16) float sm[];
    float *K = sm, *V = K + Rows<D>::FEW, *Q = V + Rows<D>::FEW, *G = Q + Rows<D>::FLOATS;
    float *P = G + Rows<D>::FLOATS, *S = P + R * PS, *lse2 = S + R * PS, *delta = lse2 + T;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, grp = a.Hq / a.Hkv / C;   // heads of this block
    const int tpc = (a.Sk + R - 1) / R;
    // window units, then the pieces of the tiles of sinks
    int piece = 0, t, kvh, b;
    unsigned x = blockIdx.x / (unsigned)C;
    if (x < (unsigned)tpc * a.B * a.Hkv) {
        t = (int)(x % (unsigned)tpc);
        x /= (unsigned)tpc;
    } else {
        x -= (unsigned)tpc * a.B * a.Hkv;
        piece = 1 + (int)(x % (unsigned)a.sp.pieces);
        x /= (unsigned)a.sp.pieces;
        t = (int)(x % (unsigned)a.sp.tiles);
        x /= (unsigned)a.sp.tiles;
    }
    kvh = (int)(x % (unsigned)a.Hkv);
    b = (int)(x / (unsigned)a.Hkv);
    const int h0 = (kvh * C + rank) * grp;
    const int ks = t * R, kl = a.Sk - ks < R ? a.Sk - ks : R;
    load_rows<D, R>(K, a.k, b, a.Sk, a.Hkv, kvh, ks, kl);
    load_rows<D, R>(V, a.v, b, a.Sk, a.Hkv, kvh, ks, kl);
    float adk[4][D / 16], adv[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) adk[i][j] = adv[i][j] = 0.f;
    const float sl2 = a.scale * LOG2E;
    WinQIter<T> it;
    if (piece == 0) it.window(a.win, a.Sq, ks, kl, h0, grp);
    else it.sinks(a.win, a.Sq, ks, h0, grp, piece - 1, a.sp.each);
    for (; it.count() > 0; it.next()) {
        const int h = it.head(), qa = it.start(), ql = it.len();
        __syncthreads();
        const float odd_q = load_rows<D, T>(Q, a.q, b, a.Sq, a.Hq, h, qa, ql) +
                            load_rows<D, T>(G, a.dout, b, a.Sq, a.Hq, h, qa, ql);
        if (threadIdx.x < T) {
            const int64_t at = ((int64_t)b * a.Hq + h) * a.Sq + qa + threadIdx.x;
            lse2[threadIdx.x] = threadIdx.x < ql ? a.lse[at] * LOG2E : 0.f;
            delta[threadIdx.x] = threadIdx.x < ql ? a.delta[at] : 0.f;
        }
        const bool odd = __syncthreads_or(odd_q != odd_q);
        float s[4][4], g[4][4];
        dots<D>(K, Q, s);
        dots<D>(V, G, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kpos = ks + ty + 8 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j, back = qa + c + a.win.off - kpos;   // how far the key lies behind the row
                const bool on = c < ql && (piece == 0 ? back >= 0 && back < a.win.window
                                                      : kpos < a.win.sinks && back >= a.win.window);
                const float p = on ? exp2f(fmaf(s[i][j], sl2, -lse2[c])) : 0.f;
                P[(ty + 8 * i) * PS + c] = p;
                S[(ty + 8 * i) * PS + c] = on ? p * (g[i][j] - delta[c]) : 0.f;
            }
        }
        __syncthreads();
        product<D>(P, G, odd, adv);
        product<D>(S, Q, odd, adk);
    }
    // the cluster's shares: each block leaves its own in shared memory (dK in Q's place, dV in
    // G's), and block `rank` adds up its part of the rows over the blocks in order
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const int at = (ty + 8 * i) * D + 4 * tx + 64 * j;
            *reinterpret_cast<float4 *>(Q + at) = make_float4(adk[i][4 * j], adk[i][4 * j + 1], adk[i][4 * j + 2], adk[i][4 * j + 3]);
            *reinterpret_cast<float4 *>(G + at) = make_float4(adv[i][4 * j], adv[i][4 * j + 1], adv[i][4 * j + 2], adv[i][4 * j + 3]);
        }
    cl.sync();
    for (int r = rank; r < kl; r += C) {
        const int kpos = ks + r;
        const bool sink = a.sp.pieces > 0 && kpos < a.win.sinks;
        if (!sink && piece != 0) continue;
        const int64_t at = (((int64_t)b * a.Sk + kpos) * a.Hkv + kvh) * D;
        float *slot = a.part + (((int64_t)b * a.Hkv + kvh) * window_part_rows(a.win, a.sp) + (int64_t)piece * 2 * a.win.sinks + kpos) * D;
        float *rk = sink ? slot : dk + at, *rv = sink ? slot + (int64_t)a.win.sinks * D : dv + at;
        for (int c = threadIdx.x; c < 2 * D; c += THREADS) {
            const bool v = c >= D;
            const int el = r * D + (v ? c - D : c);
            float sum = 0.f;
            for (int o = 0; o < C; ++o) sum += cl.map_shared_rank(v ? G : Q, o)[el];
            if (v) rv[c - D] = sum;
            else rk[c] = sum * a.scale;
        }
    }
    cl.sync();                       // the other blocks have read this one's share
}

template <int D>
constexpr int SMEM_FWD = (Rows<D>::FEW + 2 * Rows<D>::FLOATS + R * PS) * 4;
template <int D>
constexpr int SMEM_DQ = (2 * Rows<D>::FEW + 2 * Rows<D>::FLOATS + R * PS) * 4;
template <int D>
constexpr int SMEM_DKDV = (2 * Rows<D>::FEW + 2 * Rows<D>::FLOATS + 2 * R * PS + 2 * T) * 4;

template <int D>
int prepare()   // the kernels' shared memory, once per device
{
    static_assert(SMEM_DKDV<D> <= 232448, "shared memory");
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CP_ECUDA;
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return CP_OK;
    const cudaFuncAttribute what = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (cudaFuncSetAttribute(window_f32_fwd_kernel<D>, what, SMEM_FWD<D>) != cudaSuccess ||
        cudaFuncSetAttribute(window_f32_dq_kernel<D>, what, SMEM_DQ<D>) != cudaSuccess ||
        cudaFuncSetAttribute(window_f32_dkdv_kernel<D>, what, SMEM_DKDV<D>) != cudaSuccess)
        return CP_ECUDA;
    if (dev < 64) done[dev].store(true, std::memory_order_release);
    return CP_OK;
}

Args make_args(const WindowArgs &f)
{
    Args a{};
    a.B = f.B;
    a.Hq = f.Hq;
    a.Hkv = f.Hkv;
    a.Sq = f.S;
    a.Sk = f.Sk;
    a.scale = f.scale;
    a.win = f.win;
    // a few sinks begin the first tile of the window and need none of their own (5 sinks, window
    // 200: 4 tiles instead of 5)
    a.win.pack = f.win.sinks <= T / 2 ? f.win.sinks : 0;
    a.sp = window_f32_plan(a.win, a.Sq, a.Hq / a.Hkv, (int64_t)a.B * a.Hkv);
    return a;
}

template <int D>
int forward(const Args &a, float *out, float *lse, cudaStream_t st)
{
    const int rc = prepare<D>();
    if (rc) return rc;
    const int64_t units = (int64_t)((a.Sq + R - 1) / R) * a.B * a.Hq;
    if (units > 0x7fffffffLL) return CP_EUNSUPPORTED;
    window_f32_fwd_kernel<D><<<(unsigned)units, THREADS, SMEM_FWD<D>, st>>>(a, out, lse);
    return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ECUDA;
}

template <int D>
int backward(const Args &a, float *dq, float *dk, float *dv, cudaStream_t st)
{
    const int rc = prepare<D>();
    if (rc) return rc;
    const int C = window_f32_cluster(a.Hq / a.Hkv);
    const int64_t units = (int64_t)((a.Sq + R - 1) / R) * a.B * a.Hq;
    const int64_t kunits = ((int64_t)((a.Sk + R - 1) / R) + (int64_t)a.sp.tiles * a.sp.pieces) * a.B * a.Hkv * C;
    if (units > 0x7fffffffLL || kunits > 0x7fffffffLL) return CP_EUNSUPPORTED;
    const int64_t rows = (int64_t)a.B * a.Sq * a.Hq, cap = (int64_t)sm_count() * 16;
    const int64_t need = (rows + THREADS / 32 - 1) / (THREADS / 32), blocks = need < cap ? need : cap;
    window_f32_delta_kernel<D><<<(unsigned)blocks, THREADS, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return CP_ECUDA;
    window_f32_dq_kernel<D><<<(unsigned)units, THREADS, SMEM_DQ<D>, st>>>(a, dq);
    if (cudaGetLastError() != cudaSuccess) return CP_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)kunits);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_DKDV<D>;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, window_f32_dkdv_kernel<D>, a, dk, dv) != cudaSuccess) return CP_ECUDA;
    return launch_window_sinks<D>(a.part, a.win, a.sp, a.B, a.Hkv, a.Sk, dk, dv, st);
}

}  // namespace

int launch_window_fwd_f32(const float *q, const float *k, const float *v, float *out, float *lse, const WindowArgs &f,
                          cudaStream_t st)
{
    Args a = make_args(f);
    a.q = q;
    a.k = k;
    a.v = v;
    if (f.D == 64) return forward<64>(a, out, lse, st);
    if (f.D == 128) return forward<128>(a, out, lse, st);
    return CP_EUNSUPPORTED;
}

int launch_window_bwd_f32(const BwdPtrs &p, const WindowArgs &f, cudaStream_t st)
{
    Args a = make_args(f);
    a.q = static_cast<const float *>(p.q);
    a.k = static_cast<const float *>(p.k);
    a.v = static_cast<const float *>(p.v);
    a.out = static_cast<const float *>(p.out);
    a.dout = static_cast<const float *>(p.dout);
    a.lse = p.lse;
    a.delta = static_cast<float *>(p.workspace);
    a.part = a.delta + bwd_workspace_bytes(a.B, a.Hq, a.Sq) / 4;
    float *dq = static_cast<float *>(p.dq), *dk = static_cast<float *>(p.dk), *dv = static_cast<float *>(p.dv);
    if (f.D == 64) return backward<64>(a, dq, dk, dv, st);
    if (f.D == 128) return backward<128>(a, dq, dk, dv, st);
    return CP_EUNSUPPORTED;
}

}  // namespace cp
