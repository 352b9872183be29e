"""Forward of layers whose adapters have thousands of columns, or whose rows tens
of thousands: T, R^T tiles and X's slices fill the shared memory of the kernels for
few tokens, so the split, or the path, is another.  Every call the packed format
allows is computed."""
import numpy as np
import pytest
import torch

import operator_ref as ref
from gpu_util import from_dev_bf16, to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,Ns,r,tokens", [
    (384, (300,), 4096, (1, 8, 9, 16, 17, 100)),
    (4096, (512,), 2048, (16, 100, 500)),
    (1024, (256, 256), 2048, (12, 16, 40)),
    (3968, (256, 256, 512, 256, 256, 256, 256, 21), 512, (9, 17, 138)),
    (3328, (1024, 768, 59), 1000, (16, 52, 320)),
    (81280, (256,), 16, (1, 9, 16)),
    (131072, (256,), 16, (8, 16)),
    (131072, (200,), 0, (16,)),
])
def test_forward(lib, K, Ns, r, tokens):
    lis = [make_layer(LayerSpec(f"a{i}", K, n, r, 11 + 31 * i, 0.02), max(tokens)) for i, n in enumerate(Ns)]
    layer = lib.pack_grouped([to_dev(li.W) for li in lis], [to_dev(li.L) for li in lis] if r else None,
                             [to_dev(li.R) for li in lis] if r else None)
    lin = ref.Linears(lis, r)
    ws = torch.zeros(max(1, layer.workspace_bytes(max(tokens))), dtype=torch.uint8, device="cuda")
    for M in tokens:
        X = to_dev(lis[0].X[:M])
        Y = lib.linear(layer, X)
        lib.sync_status(layer)
        assert ref.rel(from_dev_bf16(Y), np.concatenate(lin.forward(ref.f64(lis[0].X[:M])), 1)) <= ref.FRO, M
        assert torch.equal(lib.linear(layer, X, ws=ws), Y)     # one workspace, sized for the most tokens
    lib.sync_status(layer)
