"""Windowed attention and the 8-bit cache without a GPU: what a call needs and what it refuses to write over."""
import pytest

from context_parallelism_02_gb300 import _lib

F32, BF16 = 0, 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,S,W,K", [(1, 8, 8, 131072, 128, 65536), (1, 32, 8, 32768, 1024, 16384), (2, 4, 4, 65536, 1, 65535),
                                            (1, 1, 1, 1048576, 16, 300000), (1, 8, 1, 8192, 64, 100), (4, 8, 8, 16384, 1024, 4)])
def test_workspace_of_many_sinks(B, Hq, Hkv, S, W, K, dtype):
    """The sinks' partial gradients in fp32 pass what K and V would take in it only by what fills the SMs: Delta,
    three times K (the slot of the window's units and pieces as long as K), and 4 x 152 units and one more per tile."""
    D = 128
    tile = 128 if dtype == BF16 else 32
    need = _lib.load().window_attn_bwd_workspace(B, Hq, Hkv, S, S, D, W, K, dtype)
    tiles = -(-K // tile) * B * Hkv
    assert need <= 256 + B * Hq * S * 4 + max(3 * B * Hkv * S * D * 4, (4 * 152 + 2 * tiles) * tile * 2 * D * 4) + 256
