"""Dense 4-bit linear on rows so long that a cluster's ranks take them in many
panels, with a chunk more or less from rank to rank."""
import numpy as np
import pytest
import torch

import operator_ref as ref
from gpu_util import from_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N,group,M", [(1015936, 16, 128, 8), (254080, 1024, 128, 16), (238208, 1000, 32, 16)])
def test_w4_uneven_ranks(lib, K, N, group, M):
    g = torch.Generator(device="cuda").manual_seed(K + N)
    W = (torch.randn(N, K, generator=g, device="cuda") * 0.02).bfloat16()
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    layer = lib.w4_pack(W, group)
    rows = np.unique(np.linspace(0, N - 1, 16).astype(int))
    w = ref.dense_w4(W[rows].view(torch.int16).cpu().numpy().view(np.uint16), group)[2]
    got = from_dev_bf16(lib.w4_linear(layer, X))[:, rows]
    lib.w4_sync_status(layer)
    assert ref.rel(got, from_dev_bf16(X) @ w.T) <= ref.FRO
