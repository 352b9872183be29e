"""Host-only refusals of slim_test_gated_timeout: slim_gated's, and a wait of
less than a microsecond."""
import ctypes

import pytest
import torch

from sparse_int4_linear_b200 import slim

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder buffers: host-only checks run where no GPU is visible")

lib = slim._lib
P = 1 << 30          # placeholder device address (never touched)


def call(L, X=2 * P, M=4, act=0, H=3 * P, GU=None, ws=4 * P, n=1 << 29, wait_us=100):
    return slim.STATUS[lib.slim_test_gated_timeout(ctypes.byref(L), X, M, act, H, GU, ws, n, wait_us, None)]


def test_refusals():
    L = slim.SlimLayerDesc()
    assert call(L) == "SLIM_ERR_STATE" and call(L, wait_us=0) == "SLIM_ERR_STATE"
    n = (ctypes.c_int32 * 2)(256, 256)
    nb = lib.slim_grouped_layer_bytes(256, 2, n, 16, 128)
    lib.slim_grouped_layer_init(ctypes.byref(L), 256, 2, n, 16, 128, P, nb, None)
    assert call(L) in ("SLIM_ERR_CUDA", "SLIM_ERR_UNSUPPORTED")    # all arguments good, no device
    assert call(L, wait_us=0) == "SLIM_ERR_ARG" and call(L, wait_us=-5) == "SLIM_ERR_ARG"
    assert call(L, act=3) == "SLIM_ERR_ARG" and call(L, X=None) == "SLIM_ERR_ARG" and call(L, M=-1) == "SLIM_ERR_ARG"
    assert call(L, ws=None) == "SLIM_ERR_WORKSPACE" and call(L, H=3 * P + 2) == "SLIM_ERR_ALIGN"
    assert call(L, M=0) == "SLIM_OK"
