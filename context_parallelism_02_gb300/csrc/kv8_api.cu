// kv8_api.cu -- the extern "C" entry points of the paged 8-bit cache (declared in
// cp.h): argument checks and dispatch.  Every check that needs no CUDA call comes first.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cp.h"
#include "kernels.h"
#include "kv8.cuh"
#include "kv_api.h"

namespace cp {

namespace {

int check_pool8(const void *cache, const float *scales, const int32_t *pages, const int32_t *lens, int B, int Hkv, int D,
                int n_pages, int page, int max_pages, Kv8Pool &p)
{
    const int rc = check_pool(cache, pages, lens, B, Hkv, D, n_pages, page, max_pages, p);
    if (rc) return rc;
    if (B > 0 && n_pages > 0 && (!scales || !aligned(scales, 4))) return CP_EINVAL;
    if ((int64_t)max_pages * page > 0x7fffffffLL - 1024) return CP_EUNSUPPORTED;   // slots are int32
    p.scales = const_cast<float *>(scales);
    return CP_OK;
}

// The bytes of the pool and the tables.
struct Sizes {
    size_t cache, scales, pages, seqs;
    Sizes(const Kv8Pool &p, int B, int D)
    {
        const size_t rows = (size_t)p.n_pages * p.Hkv * 2 << p.page_shift;
        cache = rows * D;
        scales = rows / KV8_BLOCK * 4;
        pages = (size_t)B * p.max_pages * 4;
        seqs = (size_t)B * 4;
    }
};

// From the first byte of [B][n][H][D] rows to behind the last.
size_t extent(const int64_t (&st)[3], int B, int n, int H, int D, int elem)
{
    const __int128 e = (__int128)(B - 1) * st[0] + (__int128)(n - 1) * st[1] + (__int128)(H - 1) * st[2] + D;
    return e > (__int128)1 << 56 ? (size_t)1 << 60 : (size_t)e * elem;
}

}  // namespace

}  // namespace cp

using namespace cp;

extern "C" {

int kv8_append(const void *k, const void *v, void *cache, float *scales, const int32_t *pages, const int32_t *lens,
               const int32_t *n_new, const int64_t *strides, int B, int n, int Hkv, int D, int n_pages, int page,
               int max_pages, int dtype, void *stream)
{
    NvtxScope nvtx_("kv8_append");
    Kv8AppendArgs a{};
    int rc = check_pool8(cache, scales, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (dtype != CP_F32 && dtype != CP_BF16) return CP_EUNSUPPORTED;
    if (n < 0) return CP_EINVAL;
    if (too_many(B, n, Hkv)) return CP_EUNSUPPORTED;
    if (B == 0 || n == 0) return CP_OK;
    if (!k || !v || !cache || !scales) return CP_EINVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(n_new, 4)) return CP_EINVAL;
    const int elem = dtype == CP_BF16 ? 2 : 4;
    if ((rc = set_strides(strides, n, Hkv, D, elem, a.ks)) ||
        (rc = set_strides(strides ? strides + 3 : nullptr, n, Hkv, D, elem, a.vs)))
        return rc;
    const Sizes z(a.pool, B, D);
    if (writes_over({{cache, z.cache}, {scales, z.scales}},
                    {{k, extent(a.ks, B, n, Hkv, D, elem)}, {v, extent(a.vs, B, n, Hkv, D, elem)}, {pages, z.pages},
                     {lens, z.seqs}, {n_new, z.seqs}}))
        return CP_EINVAL;
    a.k = k;
    a.v = v;
    a.n_new = n_new;
    a.B = B;
    a.n = n;
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv8_append(a, D, dtype, static_cast<cudaStream_t>(stream));
}

int kv8_gather(const void *cache, const float *scales, const int32_t *pages, const int32_t *lens, const int32_t *start,
               void *k, void *v, int B, int count, int Hkv, int D, int n_pages, int page, int max_pages, int dtype,
               void *stream)
{
    NvtxScope nvtx_("kv8_gather");
    Kv8GatherArgs a{};
    const int rc = check_pool8(cache, scales, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (dtype != CP_F32 && dtype != CP_BF16) return CP_EUNSUPPORTED;
    if (count < 0) return CP_EINVAL;
    if (too_many(B, count, Hkv)) return CP_EUNSUPPORTED;
    if (B == 0 || count == 0) return CP_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4)) return CP_EINVAL;
    const Sizes z(a.pool, B, D);
    const size_t rows = (size_t)B * count * Hkv * D * (dtype == CP_BF16 ? 2 : 4);
    if (writes_over({{k, rows}, {v, rows}}, {{cache, z.cache}, {scales, z.scales}, {pages, z.pages}, {lens, z.seqs}, {start, z.seqs}}))
        return CP_EINVAL;
    a.start = start;
    a.k = k;
    a.v = v;
    a.B = B;
    a.count = count;
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv8_gather(a, D, dtype, static_cast<cudaStream_t>(stream));
}

size_t kv8_attn_workspace(int B, int n, int Hq, int Hkv, int D, int page, int max_pages, int mass)
{
    if (B < 0 || n < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || page < 0 || max_pages < 0) return 0;
    return kv8_attn_workspace_bytes(B, n, Hq, Hkv, D, (int64_t)page * max_pages, mass != 0);
}

int kv8_attn(const void *q, const void *cache, const float *scales, const int32_t *pages, const int32_t *lens,
             const int32_t *vis, void *out, float *lse, float *mass, int B, int n, int Hq, int Hkv, int D, int n_pages,
             int page, int max_pages, int64_t window, int64_t sinks, int causal, int out_dtype, float scale,
             void *workspace, size_t ws_bytes, void *stream)
{
    NvtxScope nvtx_("kv8_attn");
    Kv8AttnArgs a{};
    int rc = check_pool8(cache, scales, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (out_dtype != CP_F32 && out_dtype != CP_BF16) return CP_EUNSUPPORTED;
    if ((rc = check_rows(q, vis, B, n, Hq, Hkv, causal, a.rows))) return rc;
    if (window < 0 || sinks < 0 || isnan(scale)) return CP_EINVAL;
    if (B == 0 || n == 0) return CP_OK;
    if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4) || !aligned(mass, 4)) return CP_EINVAL;
    const size_t need = kv8_attn_workspace(B, n, Hq, Hkv, D, page, max_pages, mass != nullptr);
    if (need == 0) return CP_EUNSUPPORTED;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < need) return CP_EINVAL;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.out = out;
    a.lse = lse;
    a.mass = mass;
    const Sizes z(a.pool, B, D);
    const size_t rows = (size_t)B * n * Hq;
    if (writes_over({{out, rows * D * (out_dtype == CP_F32 ? 4 : 2)},
                     {lse, rows * 4},
                     {mass, z.pages * page * Hkv},
                     {workspace, need}},
                    {{q, rows * D * 2}, {cache, z.cache}, {scales, z.scales}, {pages, z.pages}, {lens, z.seqs}, {vis, z.seqs * n}}))
        return CP_EINVAL;
    // no slot lies beyond the table
    const int64_t slots = (int64_t)max_pages * page;
    a.window = (int)(window > slots ? slots + 1 : window);
    a.sinks = (int)(sinks > slots ? slots : sinks);
    a.out_f32 = out_dtype == CP_F32;
    a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    a.ws = workspace;
    a.limit_ns = device_wait_limit_ns();
    a.drain_ns = device_drain_limit_ns();
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv8_attn(a, D, n_pages, static_cast<cudaStream_t>(stream));
}

int kv8_evict(void *cache, float *scales, const int32_t *pages, const int32_t *lens, const float *mass,
              const int32_t *pages_to, int32_t *kept, int32_t *lens_to, float *mass_to, int B, int Hkv, int D, int n_pages,
              int page, int max_pages, int max_to, int budget, int keep_first, int keep_last, void *stream)
{
    NvtxScope nvtx_("kv8_evict");
    Kv8EvictArgs a{};
    const int rc = check_pool8(cache, scales, pages, lens, B, Hkv, D, n_pages, page, max_pages, a.pool);
    if (rc) return rc;
    if (budget < 1 || keep_first < 0 || keep_last < 0 || keep_first > budget || keep_last > budget - keep_first)
        return CP_EINVAL;
    if (max_to < 0 || (int64_t)max_to * page < budget) return CP_EINVAL;
    if ((int64_t)max_to * page > 0x7fffffffLL - 1024) return CP_EUNSUPPORTED;
    if (B == 0) return CP_OK;
    if (!pages_to || !kept || !lens_to || !aligned(pages_to, 4) || !aligned(kept, 4) || !aligned(lens_to, 4) ||
        !aligned(mass, 4) || !aligned(mass_to, 4) || (max_pages > 0 && !mass))
        return CP_EINVAL;
    // (written while other blocks of the launch still read)
    const Sizes z(a.pool, B, D);
    const size_t to = (size_t)B * max_to * 4;
    if (writes_over({{kept, z.seqs * Hkv * budget}, {lens_to, z.seqs}, {mass_to, to * page * Hkv}},
                    {{cache, z.cache}, {scales, z.scales}, {pages, z.pages}, {lens, z.seqs}, {mass, z.pages * page * Hkv}, {pages_to, to}}))
        return CP_EINVAL;
    a.mass = mass;
    a.to = pages_to;
    a.kept = kept;
    a.lens_to = lens_to;
    a.mass_to = mass_to;
    a.B = B;
    a.max_to = max_to;
    a.budget = budget;
    a.first = keep_first;
    a.last = keep_last;
    if (!(a.pool.err = device_error_word())) return CP_ECUDA;
    return launch_kv8_evict(a, D, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
