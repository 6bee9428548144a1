// kv4.cuh -- the paged 4-bit key/value cache: its byte format, the arguments
// that its kernels share, and the device helpers that find a token block.
//
// The pool is [n_pages][Hkv][page] tokens; the tokens of one page and kv head
// are cut into blocks of 16, and a block is 20 D contiguous bytes:
//   K codes   8 D   token t: D/2 bytes at t D/2.  d = 32 gr + 8 c + o sits in the
//                   32-bit word c NG + gr of that row (NG = D/32), nibble
//                   {0,4,1,5,2,6,3,7}[o].
//   K meta    2 D   token t, group gr: fp16 scale, fp16 minimum at 4 (t NG + gr).
//   V codes   8 D   token t = 8 hf + 2 c + lo, d = 32 gr + 4 g + e: 16-bit word
//                   2 (hf 32 NG + (4 g + c) NG + gr) + lo, nibble e.
//   V meta    2 D   half hf, c, group gr: fp16 scale of tokens lo = 0, 1, then
//                   their minima, at 8 ((4 hf + c) NG + gr).
// A value is scale * code + minimum.  The orders are those of the A operand of
// mma.m16n8k16: a lane's 32-bit words hold pairs (k, k+1) of one row in their
// low and high halves, so a code pair becomes an fp16 pair by one mask, and a
// lane's share of a block is contiguous (16-byte shared-memory reads at D = 128).
// Every code word and meta word belongs to one token in whole 2- or 4-byte
// units, so tokens are written without reading their neighbours.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cp_common.cuh"

namespace cp {

constexpr int KV4_BLOCK = 16;   // tokens of a block
constexpr int KV4_GROUP = 32;   // elements that share a scale and a minimum

template <int D>
struct Kv4 {
    static constexpr int NG = D / KV4_GROUP;
    static constexpr int K_META = 8 * D;
    static constexpr int V_CODES = 10 * D;
    static constexpr int V_META = 18 * D;
    static constexpr int BYTES = 20 * D;
};

// A pool and the page table of a batch.
struct Kv4Pool {
    uint8_t *data;          // [n_pages][Hkv][page / 16][20 D]
    const int32_t *pages;   // [B][max_pages]
    const int32_t *lens;    // [B] tokens in the cache
    int n_pages, max_pages, page_shift, Hkv;
    unsigned *err;          // device error word
};

#if defined(__CUDACC__)

__device__ __forceinline__ void kv4_report(unsigned *err) { atomicCAS(err, 0u, ERRW_CACHE); }

// Physical page of logical page lp of sequence b; -1 (and CP_ECACHE in the
// error word) if the table has no valid entry there.
__device__ __forceinline__ int kv4_page(const Kv4Pool &c, int b, int64_t lp)
{
    int id = -1;
    if (lp >= 0 && lp < c.max_pages) id = c.pages[(int64_t)b * c.max_pages + lp];
    if (id < 0 || id >= c.n_pages) {
        kv4_report(c.err);
        return -1;
    }
    return id;
}

// Block of 16 tokens number blk within physical page id, kv head h.
template <int D>
__device__ __forceinline__ uint8_t *kv4_block(const Kv4Pool &c, int id, int h, int blk)
{
    return c.data + ((((int64_t)id * c.Hkv + h) << (c.page_shift - 4)) + blk) * Kv4<D>::BYTES;
}

// Every kernel of the cache is launched so that its blocks may start while the
// kernel before it on the stream ends (kv4_launch).  kv4_trigger lets its own successor
// do the same, as soon as every block has called it; behind kv4_wait the kernel before
// it is complete and its writes are visible.  A kernel that triggers first says nothing
// about its predecessors: its successor must wait before it reads anything.
// What the kernels read may be written while they are already resident, so no load takes
// the read-only path (ld.global.nc asks for data that nobody writes while the kernel
// lives, and is not ordered behind the wait); plain loads are.
__device__ __forceinline__ void kv4_trigger() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void kv4_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void kv4_begin()
{
    kv4_trigger();
    kv4_wait();
}

// Length of sequence b, held inside the page table's reach.  EARLY: by a kernel that has
// not waited yet, whose predecessor triggered behind its own wait.
template <bool EARLY = false>
__device__ __forceinline__ int kv4_len(const Kv4Pool &c, int b)
{
    const int64_t cap = (int64_t)c.max_pages << c.page_shift;
    int got;
    if (EARLY) asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(got) : "l"(c.lens + b) : "memory");
    else got = c.lens[b];
    int64_t len = got;
    if (len < 0 || len > cap) {
        kv4_report(c.err);
        len = len < 0 ? 0 : cap;
    }
    return (int)len;
}

#endif

template <typename... P, typename... A>
inline cudaError_t kv4_launch(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Kv4AppendArgs {
    Kv4Pool pool;            // lens: tokens before the append
    const void *k, *v, *q;
    void *q_out;             // [B][n][Hq][D] or null
    __nv_bfloat16 *summary;  // [n_pages][Hkv][2][D] or null
    const int32_t *n_new, *positions;   // [B], [B][n], or null
    const float *cos, *sin;  // [max_pos][rot / 2]
    int64_t ks[3], vs[3], qs[3];        // element strides of batch, token, head
    int B, n, Hq, rot, interleaved, max_pos;
};
int launch_kv4_append(const Kv4AppendArgs &a, int D, int dtype, cudaStream_t st);

struct Kv4GatherArgs {
    Kv4Pool pool;
    const int32_t *start;    // [B] or null (0)
    void *k, *v;             // [B][count][Hkv][D]
    int B, count;
};
int launch_kv4_gather(const Kv4GatherArgs &a, int D, int dtype, cudaStream_t st);

// What a query row sees: slots below vis[b][j] where vis is given, else below
// len - (n - 1) + j (causal) or len.
struct Kv4Rows {
    const int32_t *vis;
    int B, n, Hq, causal;
};

#if defined(__CUDACC__)
__device__ __forceinline__ int kv4_limit(const Kv4Rows &r, int b, int j, int len)
{
    int64_t lim = len;
    if (r.vis) lim = r.vis[(int64_t)b * r.n + j];
    else if (r.causal) lim = (int64_t)len - (r.n - 1) + j;
    return (int)(lim < 0 ? 0 : lim > len ? len : lim);
}
#endif

struct Kv4AttnArgs {
    Kv4Pool pool;
    Kv4Rows rows;
    const __nv_bfloat16 *q;  // [B][n][Hq][D]
    const int32_t *sel;      // [B][n][Hkv][n_sel] or null
    void *out;               // [B][n][Hq][D]
    float *lse;              // [B][Hq][n]
    int n_sel, out_f32;
    float scale;
    void *ws;
    uint64_t limit_ns, drain_ns;
};
size_t kv4_attn_workspace_bytes(int D);
int launch_kv4_attn(const Kv4AttnArgs &a, int D, cudaStream_t st);

struct Kv4SelectArgs {
    Kv4Pool pool;            // data unused
    Kv4Rows rows;
    const __nv_bfloat16 *q, *summary;
    int32_t *sel;            // [B][n][Hkv][n_sel]
    float *scores;           // [B][n][Hkv][max_pages]
    int n_sel, keep_first, keep_last;
};
int launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st);

}  // namespace cp
