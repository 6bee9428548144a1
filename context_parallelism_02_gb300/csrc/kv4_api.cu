// kv4_api.cu -- the extern "C" entry points of the paged 4-bit cache (declared
// in cp.h): argument checks and dispatch.  Every check that needs no CUDA call
// comes first.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "cp.h"
#include "kernels.h"
#include "kv4.cuh"

namespace cp {

namespace {

struct NvtxScope {
    explicit NvtxScope(const char *name) { nvtxRangePushA(name); }
    ~NvtxScope() { nvtxRangePop(); }
    NvtxScope(const NvtxScope &) = delete;
    NvtxScope &operator=(const NvtxScope &) = delete;
};

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Sizes that every call has; fills the pool except data and err.
int check_pool(const void *cache, const int32_t *pages, const int32_t *lens, int B, int Hkv, int D,
               int n_pages, int page, int max_pages, Kv4Pool &p)
{
    if (B < 0 || Hkv < 1 || n_pages < 0 || max_pages < 0) return CP_EINVAL;
    if (D != 64 && D != 128) return CP_EUNSUPPORTED;
    int shift = 4;
    while (shift < 8 && (1 << shift) != page) ++shift;
    if ((1 << shift) != page) return CP_EUNSUPPORTED;
    if (B > 0 && (!pages || !lens || !aligned(pages, 4) || !aligned(lens, 4))) {
        if (!lens || max_pages > 0) return CP_EINVAL;
        if (!aligned(lens, 4)) return CP_EINVAL;
    }
    if (B > 0 && n_pages > 0 && (!cache || !aligned(cache, 16))) return CP_EINVAL;
    p.data = static_cast<uint8_t *>(const_cast<void *>(cache));
    p.pages = pages;
    p.lens = lens;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.page_shift = shift;
    p.Hkv = Hkv;
    p.err = nullptr;
    return CP_OK;
}

// Element strides (batch, token, head) of a [B][n][H][D] tensor whose rows are
// contiguous; rows must start on 16-byte boundaries.
int set_strides(const int64_t *given, int n, int H, int D, int elem, int64_t (&s)[3])
{
    if (!given) {
        s[0] = (int64_t)n * H * D;
        s[1] = (int64_t)H * D;
        s[2] = D;
        return CP_OK;
    }
    for (int i = 0; i < 3; ++i) {
        if (given[i] < 0 || given[i] % (16 / elem)) return CP_EINVAL;
        s[i] = given[i];
    }
    return CP_OK;
}

// Whether [B][n][heads] rows are more than the launches count in 64 bits (far more than any
// memory holds: rows with strides of 0 need none).
bool too_many(int B, int n, int heads)
{
    return (unsigned __int128)(unsigned)B * (unsigned)n * (unsigned)heads > (unsigned __int128)1 << 48;
}

int check_rows(const void *q, const int32_t *vis, int B, int n, int Hq, int Hkv, int causal, Kv4Rows &r)
{
    if (B < 0 || n < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (causal != 0 && causal != 1)) return CP_EINVAL;
    if (too_many(B, n, Hq)) return CP_EUNSUPPORTED;
    if (B > 0 && n > 0 && (!q || !aligned(q, 16) || !aligned(vis, 4))) return CP_EINVAL;
    r.vis = vis;
    r.B = B;
    r.n = n;
    r.Hq = Hq;
    r.causal = causal;
    return CP_OK;
}

}  // namespace

}  // namespace cp

using namespace cp;

extern "C" {

int kv4_append(const void *k, const void *v, const void *q, void *q_out, void *cache, void *summary,
               const int32_t *pages, const int32_t *lens, const int32_t *n_new,
               const int32_t *positions, const float *cosine, const float *sine,
               const int64_t *strides, int B, int n, int Hq, int Hkv, int D, int n_pages, int page,
               int max_pages, int rot, int interleaved, int max_pos, int dtype, void *stream)
{
    NvtxScope nvtx_("kv4_append");
    Kv4AppendArgs a{};
    int rc = check_pool(cache, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (dtype != CP_F32 && dtype != CP_BF16) return CP_EUNSUPPORTED;
    if (n < 0 || (!q) != (!q_out) || (q && Hq < 1) || (interleaved != 0 && interleaved != 1)) return CP_EINVAL;
    if (q && Hq % Hkv) return CP_EINVAL;
    if (rot < 0 || rot > D || rot % 16 || max_pos < 0) return CP_EINVAL;
    if (too_many(B, n, Hkv) || (q && too_many(B, n, Hq))) return CP_EUNSUPPORTED;
    if (B == 0 || n == 0) return CP_OK;
    if (!k || !v || !cache) return CP_EINVAL;
    if (rot && (!cosine || !sine || !aligned(cosine, 16) || !aligned(sine, 16))) return CP_EINVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(summary, 16) ||
        !aligned(n_new, 4) || !aligned(positions, 4))
        return CP_EINVAL;
    const int elem = dtype == CP_BF16 ? 2 : 4;
    if ((rc = set_strides(strides, n, Hkv, D, elem, a.ks)) ||
        (rc = set_strides(strides ? strides + 3 : nullptr, n, Hkv, D, elem, a.vs)) ||
        (rc = set_strides(strides && q ? strides + 6 : nullptr, n, q ? Hq : 1, D, elem, a.qs)))
        return rc;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.summary = static_cast<__nv_bfloat16 *>(summary);
    a.n_new = n_new;
    a.positions = positions;
    a.cos = cosine;
    a.sin = sine;
    a.B = B;
    a.n = n;
    a.Hq = q ? Hq : 1;
    a.rot = rot;
    a.interleaved = interleaved;
    a.max_pos = max_pos;
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv4_append(a, D, dtype, static_cast<cudaStream_t>(stream));
}

int kv4_gather(const void *cache, const int32_t *pages, const int32_t *lens, const int32_t *start,
               void *k, void *v, int B, int count, int Hkv, int D, int n_pages, int page,
               int max_pages, int dtype, void *stream)
{
    NvtxScope nvtx_("kv4_gather");
    Kv4GatherArgs a{};
    const int rc = check_pool(cache, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (dtype != CP_F32 && dtype != CP_BF16) return CP_EUNSUPPORTED;
    if (count < 0) return CP_EINVAL;
    if (too_many(B, count, Hkv)) return CP_EUNSUPPORTED;
    if (B == 0 || count == 0) return CP_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4)) return CP_EINVAL;
    a.start = start;
    a.k = k;
    a.v = v;
    a.B = B;
    a.count = count;
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv4_gather(a, D, dtype, static_cast<cudaStream_t>(stream));
}

size_t kv4_attn_workspace(int D) { return kv4_attn_workspace_bytes(D); }

int kv4_attn(const void *q, const void *cache, const int32_t *pages, const int32_t *lens,
             const int32_t *vis, const int32_t *sel, void *out, float *lse, int B, int n, int Hq,
             int Hkv, int D, int n_pages, int page, int max_pages, int n_sel, int causal,
             int out_dtype, float scale, void *workspace, size_t ws_bytes, void *stream)
{
    NvtxScope nvtx_("kv4_attn");
    Kv4AttnArgs a{};
    int rc = check_pool(cache, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (out_dtype != CP_F32 && out_dtype != CP_BF16) return CP_EUNSUPPORTED;
    if ((rc = check_rows(q, vis, B, n, Hq, Hkv, causal, a.rows))) return rc;
    if (sel ? n_sel < 1 || !aligned(sel, 4) : n_sel != 0) return CP_EINVAL;
    if (n_sel > 1 << 26) return CP_EUNSUPPORTED;   // blocks of 16 tokens are counted in 32 bits
    if (isnan(scale)) return CP_EINVAL;
    if (B == 0 || n == 0) return CP_OK;
    if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return CP_EINVAL;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < kv4_attn_workspace_bytes(D)) return CP_EINVAL;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.sel = sel;
    a.out = out;
    a.lse = lse;
    a.n_sel = n_sel;
    a.out_f32 = out_dtype == CP_F32;
    a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    a.ws = workspace;
    a.limit_ns = device_wait_limit_ns();
    a.drain_ns = device_drain_limit_ns();
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv4_attn(a, D, static_cast<cudaStream_t>(stream));
}

size_t kv4_select_workspace(int B, int n, int Hkv, int max_pages)
{
    if (B < 0 || n < 0 || Hkv < 1 || max_pages < 0) return 0;
    const unsigned __int128 b = (unsigned __int128)(unsigned)B * (unsigned)n * (unsigned)Hkv * (unsigned)max_pages * 4u;
    if (b > ((unsigned __int128)1 << 62)) return 0;
    const size_t s = ((size_t)b + 255) / 256 * 256;
    return s ? s : 256;
}

int kv4_select(const void *q, const void *summary, const int32_t *pages, const int32_t *lens,
               const int32_t *vis, int32_t *sel, int B, int n, int Hq, int Hkv, int D, int n_pages,
               int page, int max_pages, int n_sel, int causal, int keep_first, int keep_last,
               void *workspace, size_t ws_bytes, void *stream)
{
    NvtxScope nvtx_("kv4_select");
    Kv4SelectArgs a{};
    int rc = check_pool(summary, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if ((rc = check_rows(q, vis, B, n, Hq, Hkv, causal, a.rows))) return rc;
    if (n_sel < 1 || keep_first < 0 || keep_last < 0 || keep_first > n_sel || keep_last > n_sel - keep_first)
        return CP_EINVAL;
    if (B == 0 || n == 0) return CP_OK;
    const size_t need = kv4_select_workspace(B, n, Hkv, max_pages);
    if (!sel || !aligned(sel, 4)) return CP_EINVAL;
    if (need == 0 || !workspace || !aligned(workspace, 16) || ws_bytes < need) return CP_EINVAL;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.summary = static_cast<const __nv_bfloat16 *>(summary);
    a.sel = sel;
    a.scores = static_cast<float *>(workspace);
    a.n_sel = n_sel;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.pool.data = nullptr;
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv4_select(a, D, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
