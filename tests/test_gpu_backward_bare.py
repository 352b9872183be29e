"""Gradients of an adapter that a layer does not have are None, asked for alone
as well."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_adapter_gradients_of_a_layer_without_one(lib):
    g = torch.Generator().manual_seed(1)
    W = [(torch.randn(256, 256, generator=g) * 0.02).bfloat16().cuda() for _ in range(2)]
    layer = lib.pack_grouped(W)
    X = torch.ones(5, 256, dtype=torch.bfloat16, device="cuda")
    dY = torch.ones(5, 512, dtype=torch.bfloat16, device="cuda")
    for need in (("dL", "dR"), ("dL",), ["dR"]):
        assert lib.linear_backward(layer, X, dY, need=need) == (None, None, None)
        assert lib.gated_backward(layer, X, dY, X, need=need) == (None, None, None)
    dX, dL, dR = lib.linear_backward(layer, X, dY, need=("dX", "dL"))
    assert dX.shape == (5, 256) and dL is None and dR is None
    with pytest.raises(ValueError):
        lib.linear_backward(layer, X, dY[:, :256], need=("dL",))
    with pytest.raises(lib.SlimError):
        lib.linear_backward(layer, X, dY, need=())
