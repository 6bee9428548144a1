// window_api.cu -- the extern "C" entry points of windowed attention with sinks
// (declared in cp.h): argument checks and dispatch.  Every check that needs no CUDA
// call comes first.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cp.h"
#include "kernels.h"
#include "kv_api.h"

namespace cp {

namespace {

bool aligned16(const void *p) { return aligned(p, 16); }

// Checks what the windowed calls share and fills the arguments; 1: nothing to do.
int window_args(int B, int Hq, int Hkv, int64_t Sq, int64_t Sk, int D, int64_t window, int64_t sinks, int dtype,
                float scale, WindowArgs &a)
{
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || Sq < 0 || Sk < Sq || window < 1 || sinks < 0 || isnan(scale))
        return CP_EINVAL;
    if (dtype != CP_F32 && dtype != CP_BF16) return CP_EUNSUPPORTED;
    if (D != 64 && D != 128) return CP_EUNSUPPORTED;
    if (Sk > 0x7fffffffLL - 1024) return CP_EUNSUPPORTED;   // positions and tile ends are int32
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.S = (int)Sq;
    a.Sk = (int)Sk;
    a.D = D;
    a.N = 1;
    a.causal = 1;
    a.layout = CP_LAYOUT_CONTIGUOUS;
    a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    a.rank_lo = 0;
    a.rank_hi = 1;
    a.upc = 0;
    a.head_grouped = 0;
    a.n_units = 0;
    a.err = nullptr;
    a.limit_ns = device_wait_limit_ns();
    a.drain_ns = device_drain_limit_ns();
    a.win.off = (int)(Sk - Sq);
    a.win.window = (int)(window < Sk ? window : Sk < 1 ? 1 : Sk);
    a.win.sinks = (int)(sinks < Sk ? sinks : Sk);
    a.win.pack = window_pack(a.win.sinks);
    return B == 0 || Sk == 0 ? 1 : CP_OK;
}

}  // namespace

}  // namespace cp

using namespace cp;

extern "C" {

int window_attn_fwd(const void *q, const void *k, const void *v, void *out, float *lse, int B, int Hq, int Hkv,
                    int64_t Sq, int64_t Sk, int D, int64_t window, int64_t sinks, int dtype, float scale, void *stream)
{
    NvtxScope nvtx_("window_attn_fwd");
    WindowArgs a;
    const int rc = window_args(B, Hq, Hkv, Sq, Sk, D, window, sinks, dtype, scale, a);
    if (rc < 0) return rc;
    if (rc || Sq == 0) return CP_OK;
    if (!q || !k || !v || !out || !lse) return CP_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || ((uintptr_t)lse & 3u)) return CP_EINVAL;
    const size_t row = (size_t)B * D * (dtype == CP_BF16 ? 2 : 4), nq = row * Sq * Hq, nk = row * Sk * Hkv;
    if (writes_over({{out, nq}, {lse, (size_t)B * Hq * Sq * 4}}, {{q, nq}, {k, nk}, {v, nk}})) return CP_EINVAL;
    if (!(a.err = device_error_word())) return CP_ECUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == CP_F32)
        return launch_window_fwd_f32(static_cast<const float *>(q), static_cast<const float *>(k),
                                     static_cast<const float *>(v), static_cast<float *>(out), lse, a, st);
    return launch_window_fwd_bf16(q, k, v, out, lse, a, st);
}

size_t window_attn_bwd_workspace(int B, int Hq, int Hkv, int64_t Sq, int64_t Sk, int D, int64_t window, int64_t sinks,
                                 int dtype)
{
    WindowArgs a;
    if (window_args(B, Hq, Hkv, Sq, Sk, D, window, sinks, dtype, 1.f, a) < 0) return 0;
    const size_t b = window_bwd_workspace_bytes(B, Hq, Hkv, a.S, D, dtype, a.win);
    return b ? b : 256;
}

int window_attn_bwd(const void *q, const void *k, const void *v, const void *out, const float *lse, const void *dout,
                    void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int64_t Sq, int64_t Sk, int D,
                    int64_t window, int64_t sinks, int dtype, float scale, void *workspace, size_t ws_bytes,
                    void *stream)
{
    NvtxScope nvtx_("window_attn_bwd");
    WindowArgs a;
    const int rc = window_args(B, Hq, Hkv, Sq, Sk, D, window, sinks, dtype, scale, a);
    if (rc < 0) return rc;
    if (rc) return CP_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!k || !v || !dk || !dv || !aligned16(k) || !aligned16(v) || !aligned16(dk) || !aligned16(dv)) return CP_EINVAL;
    const size_t row = (size_t)B * D * (dtype == CP_BF16 ? 2 : 4), nq = row * Sq * Hq, nk = row * Sk * Hkv;
    if (Sq == 0) {   // no row sees the keys
        if (writes_over({{dk, nk}, {dv, nk}}, {{k, nk}, {v, nk}})) return CP_EINVAL;
        return cudaMemsetAsync(dk, 0, nk, st) == cudaSuccess && cudaMemsetAsync(dv, 0, nk, st) == cudaSuccess ? CP_OK
                                                                                                                : CP_ECUDA;
    }
    if (!q || !out || !lse || !dout || !dq || !workspace) return CP_EINVAL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(dout) || !aligned16(dq) || !aligned16(workspace) ||
        ((uintptr_t)lse & 3u))
        return CP_EINVAL;
    const size_t need = window_bwd_workspace_bytes(B, Hq, Hkv, a.S, D, dtype, a.win);
    if (ws_bytes < need) return CP_EINVAL;
    const BwdPtrs p{q, k, v, out, lse, dout, dq, dk, dv, workspace};
    if (writes_over({{dq, nq}, {dk, nk}, {dv, nk}, {workspace, need}},
                    {{q, nq}, {k, nk}, {v, nk}, {out, nq}, {dout, nq}, {lse, (size_t)B * Hq * Sq * 4}}))
        return CP_EINVAL;
    if (!(a.err = device_error_word())) return CP_ECUDA;
    if (dtype == CP_F32) return launch_window_bwd_f32(p, a, st);
    return launch_window_bwd_bf16(p, a, st);
}

}  // extern "C"
