"""Windowed attention on the CPU: the walks of the kernels, and what the calls refuse."""
import ctypes
import os
import subprocess

import pytest

from context_parallelism_02_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_walks_cover_the_visible_pairs_once(tmp_path):
    """WinIter and WinQIter with the masks that the kernels apply: every visible pair once."""
    exe = tmp_path / "walk"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(ROOT, "tests", "window_walk_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def _fwd(**kw):
    a = dict(p=None, B=1, Hq=2, Hkv=1, Sq=64, Sk=64, D=64, window=8, sinks=2, dtype=1, scale=-1.0) | kw
    return _lib.load().window_attn_fwd(*[a["p"]] * 5, a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Sk"], a["D"], a["window"],
                                       a["sinks"], a["dtype"], a["scale"], None)


def _bwd(ws=None, n=0, **kw):
    a = dict(p=None, B=1, Hq=2, Hkv=1, Sq=64, Sk=64, D=64, window=8, sinks=2, dtype=1, scale=-1.0) | kw
    return _lib.load().window_attn_bwd(*[a["p"]] * 9, a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Sk"], a["D"], a["window"],
                                       a["sinks"], a["dtype"], a["scale"], ws, n, None)


BAD = [(dict(), _lib.CP_EINVAL), (dict(Hq=3, Hkv=2), _lib.CP_EINVAL), (dict(window=0), _lib.CP_EINVAL),
       (dict(sinks=-1), _lib.CP_EINVAL), (dict(Sq=65), _lib.CP_EINVAL), (dict(Sq=-1), _lib.CP_EINVAL),
       (dict(B=-1), _lib.CP_EINVAL), (dict(Hkv=0), _lib.CP_EINVAL), (dict(scale=float("nan")), _lib.CP_EINVAL),
       (dict(D=96), _lib.CP_EUNSUPPORTED), (dict(dtype=2), _lib.CP_EUNSUPPORTED),
       (dict(Sk=2 ** 31 - 1000), _lib.CP_EUNSUPPORTED), (dict(Sk=2 ** 40), _lib.CP_EUNSUPPORTED),
       (dict(p=ctypes.c_void_p(8)), _lib.CP_EINVAL)]


@pytest.mark.parametrize("kw,code", BAD)
def test_refused_before_any_cuda_call(kw, code):
    assert _fwd(**kw) == code
    assert _bwd(**kw) == code


def test_empty_calls_and_workspace():
    L = _lib.load()
    assert _fwd(B=0) == _lib.CP_OK and _fwd(Sq=0) == _lib.CP_OK and _fwd(Sq=0, Sk=0) == _lib.CP_OK
    assert _bwd(B=0) == _lib.CP_OK and _bwd(Sq=0, Sk=0) == _lib.CP_OK
    p = ctypes.c_void_p(16)
    need = L.window_attn_bwd_workspace(1, 2, 1, 64, 64, 64, 8, 2, 1)
    assert need >= 2 * 64 * 4
    assert _bwd(p=p, ws=p, n=need - 1) == _lib.CP_EINVAL
    assert _bwd(p=p, ws=None, n=need) == _lib.CP_EINVAL
    assert _bwd(p=p, ws=ctypes.c_void_p(24), n=need) == _lib.CP_EINVAL
    assert L.window_attn_bwd_workspace(1, 2, 1, 64, 64, 96, 8, 2, 1) == 0
    assert L.window_attn_bwd_workspace(1, 2, 1, 64, 64, 64, 0, 2, 1) == 0
    # the sinks' partial sums grow with the rows behind their window, not with the rows squared
    a, b = (L.window_attn_bwd_workspace(1, 8, 8, S, S, 128, 1024, 4, 1) for S in (65536, 131072))
    assert a < b <= 2.1 * a
