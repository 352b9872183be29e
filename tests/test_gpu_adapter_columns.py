"""T = X L over several column blocks of 256, whose last one is narrower: every
width from 16 to 256, for the forward and the gated block, with enough tokens
for blocks of 256 (over 512, or many adapter columns) and with fewer."""
import numpy as np
import pytest

import operator_ref as ref
from gpu_util import from_dev_bf16, to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [40, 600])
@pytest.mark.parametrize("r", [264, 330, 384, 400, 448, 512, 640, 700, 704, 960, 1024])
def test_linear_ranks_beyond_one_block(lib, r, M):
    li = make_layer(LayerSpec("c", 512, 300, r, 7 + r, 0.02), M)
    layer = lib.pack(to_dev(li.W), to_dev(li.L), to_dev(li.R))
    Y = lib.linear(layer, to_dev(li.X))
    lib.sync_status(layer)
    assert ref.rel(from_dev_bf16(Y), ref.Linears([li], r).forward(ref.f64(li.X))[0]) <= ref.FRO


@pytest.mark.parametrize("r", [130, 160, 192, 214, 224, 320, 352, 480])
def test_gated_ranks_beyond_one_block(lib, r):
    M, F = 600, 256
    lis = [make_layer(LayerSpec(f"c{i}", 384, F, r, 9 + r + 31 * i, 0.02), M) for i in range(2)]
    layer = lib.pack_grouped(*([to_dev(getattr(li, k)) for li in lis] for k in "WLR"))
    G, U = ref.Linears(lis, r).forward(ref.f64(lis[0].X))
    H, GU = lib.gated(layer, to_dev(lis[0].X), keep=True)
    lib.sync_status(layer)
    assert ref.rel(from_dev_bf16(H), ref.act("silu", G) * U) <= ref.FRO
    assert ref.rel(from_dev_bf16(GU), np.concatenate([G, U], 1)) <= ref.FRO
