// kv_api.h -- argument checks that the entry points of the paged caches (and of windowed
// attention) share.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include <nvtx3/nvToolsExt.h>

#include "cp.h"
#include "kv4.cuh"

namespace cp {

namespace {

struct NvtxScope {
    explicit NvtxScope(const char *name) { nvtxRangePushA(name); }
    ~NvtxScope() { nvtxRangePop(); }
    NvtxScope(const NvtxScope &) = delete;
    NvtxScope &operator=(const NvtxScope &) = delete;
};

inline bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Whether two buffers share a byte; null buffers do not.
inline bool overlap(const void *p, size_t np, const void *q, size_t nq)
{
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return np && nq && p && q && a < b + nq && b < a + np;
}

// Whether one of the buffers that a call writes shares a byte with one that it reads, or with
// another that it writes.
struct Buffer {
    const void *p;
    size_t bytes;
};
inline bool writes_over(std::initializer_list<Buffer> writes, std::initializer_list<Buffer> reads)
{
    for (const Buffer *w = writes.begin(); w != writes.end(); ++w) {
        for (const Buffer *x = writes.begin(); x != w; ++x)
            if (overlap(w->p, w->bytes, x->p, x->bytes)) return true;
        for (const Buffer &r : reads)
            if (overlap(w->p, w->bytes, r.p, r.bytes)) return true;
    }
    return false;
}

// Sizes that every call has; fills the pool except data and err.
inline int check_pool(const void *cache, const int32_t *pages, const int32_t *lens, int B, int Hkv, int D,
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
inline int set_strides(const int64_t *given, int n, int H, int D, int elem, int64_t (&s)[3])
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
inline bool too_many(int B, int n, int heads)
{
    return (unsigned __int128)(unsigned)B * (unsigned)n * (unsigned)heads > (unsigned __int128)1 << 48;
}

inline int check_rows(const void *q, const int32_t *vis, int B, int n, int Hq, int Hkv, int causal, Kv4Rows &r)
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
