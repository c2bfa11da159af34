"""The delta rule's workspaces: as large as the header says, for many short sequences too (CPU)."""
import ctypes

import pytest

from depthwise_causal_short_gb300 import _build, attn


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return attn.load()


@pytest.mark.parametrize("total,nseq,Hk,Hv,K,V", [
    (16384, 2, 8, 16, 128, 128), (4096, 4096, 8, 16, 128, 128), (0, 7, 1, 1, 8, 8), (1, 1, 1, 1, 8, 8), (64, 1, 8, 8, 128, 128),
    (3108, 7, 4, 4, 64, 96), (100000, 3, 4, 32, 64, 256), (5000, 2000, 2, 6, 40, 56), (513, 1, 1, 2, 32, 32),
])
def test_sizes(lib, total, nseq, Hk, Hv, K, V):
    n = ctypes.c_size_t(0)
    tiles, chunks = (V + 31) // 32, (total // 64 + nseq) * Hv if total else 0
    slack = 16 * 256 + 2 * (1 << 16) * Hv * tiles  # the parts' alignment, the last part of 512 tokens
    assert lib.cattn_delta_fwd_workspace_bytes(total, nseq, Hk, Hv, K, V, ctypes.byref(n)) == 0
    assert chunks * 48 * 1024 <= n.value <= chunks * 49 * 1024 + slack
    assert lib.cattn_delta_bwd_workspace_bytes(total, nseq, Hk, Hv, K, V, ctypes.byref(n)) == 0
    tile = 66 if nseq * Hv * tiles <= 96 else 56
    assert n.value <= chunks * (49 + tile * tiles) * 1024 + slack
