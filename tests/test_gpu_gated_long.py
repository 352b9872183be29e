"""Gated block for few tokens on rows longer than the adapter kernel can stage
(81,152 columns, 162,304 up to 8 tokens): on both sides of those lengths."""
import numpy as np
import pytest

import operator_ref as ref
from gpu_util import from_dev_bf16, to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,M", [(81152, 9), (81280, 9), (81280, 20), (162304, 8), (162432, 1), (162432, 8)])
def test_gated_long_rows_with_an_adapter(lib, K, M, F=256, r=20):
    lis = [make_layer(LayerSpec(f"l{i}", K, F, r, 7 + 31 * i, 0.02), M) for i in range(2)]
    layer = lib.pack_grouped(*([to_dev(getattr(li, k)) for li in lis] for k in "WLR"))
    X = to_dev(lis[0].X)
    rows = np.arange(0, F, 15)
    for li in lis:      # (every row's definition would take a while in 64 bits)
        li.W, li.R = np.ascontiguousarray(li.W[rows]), np.ascontiguousarray(li.R[:, rows])
    G, U = ref.Linears(lis, r).forward(ref.f64(lis[0].X))
    H, GU = lib.gated(layer, X, keep=True)
    lib.sync_status(layer)
    assert ref.rel(from_dev_bf16(H)[:, rows], ref.act("silu", G) * U) <= ref.FRO
    assert ref.rel(from_dev_bf16(GU)[:, rows], G) <= ref.FRO
    assert ref.rel(from_dev_bf16(GU)[:, F + rows], U) <= ref.FRO
    assert (lib.gated(layer, X) == H).all()
