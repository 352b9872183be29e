"""Workspace queries of layers with thousands of adapter columns or long rows
(host only): a workspace sized for M serves every smaller M, on whatever path."""
import ctypes

import pytest
import torch

from sparse_int4_linear_b200 import slim

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder buffers: host-only checks run where no GPU is visible")

lib = slim._lib


@pytest.mark.parametrize("G,r", [(1, 1024), (1, 2048), (1, 4096), (2, 1000), (2, 2048), (3, 1000), (8, 512), (4, 16), (1, 0)])
@pytest.mark.parametrize("K", [128, 1024, 4096, 11008, 131072])
def test_workspace_never_decreases(G, r, K):
    L = slim.SlimLayerDesc()
    n = (ctypes.c_int32 * G)(*[256] * G)
    nb = lib.slim_grouped_layer_bytes(K, G, n, r, 128)
    assert nb > 0
    lib.slim_grouped_layer_init(ctypes.byref(L), K, G, n, r, 128, 1 << 30, nb, None)
    sizes = [lib.slim_workspace_bytes(ctypes.byref(L), M) for M in (1, 2, 7, 8, 9, 12, 16, 17, 40, 100, 300, 1000, 4096, 16384)]
    assert sizes == sorted(sizes)
    assert all(lib.slim_linear_launches(ctypes.byref(L), M) > 0 for M in (1, 8, 9, 16, 17, 4096))
