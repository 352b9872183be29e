"""A workspace that is not one piece of the layer's device memory is refused
before its address reaches a kernel."""
from types import SimpleNamespace

import pytest
import torch

from sparse_int4_linear_b200 import slim


def test_a_host_workspace_is_refused():
    layer = SimpleNamespace(device=torch.device("cuda", 0), device_index=0)
    for ws in (torch.zeros(4096, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8).expand(4096)):
        with pytest.raises(ValueError):
            slim._scratch(ws, layer)


def test_address_and_bytes():
    """Bytes are counted whatever the element type (a CPU stand-in for the layer's device, index -1)."""
    layer = SimpleNamespace(device=torch.device("cpu"), device_index=-1)
    ws = torch.zeros(1024, dtype=torch.float32)
    assert slim._scratch(ws, layer) == (ws.data_ptr(), 4096)
    for bad in (ws[::2], ws[:1].expand(1024)):
        with pytest.raises(ValueError):
            slim._scratch(bad, layer)


@pytest.mark.gpu
def test_every_call_refuses_it(lib):
    g = torch.Generator().manual_seed(1)
    W = [(torch.randn(256, 256, generator=g) * 0.02).bfloat16().cuda() for _ in range(2)]
    layer, q4 = lib.pack_grouped(W), lib.w4_pack(W[0])
    X = torch.zeros(600, 256, dtype=torch.bfloat16, device="cuda")
    dY, dH = torch.zeros(600, 512, dtype=torch.bfloat16, device="cuda"), X.clone()
    host = torch.zeros(1 << 24, dtype=torch.uint8)
    spread = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 24)
    for ws in (host, spread):
        for call in (lambda: lib.gated(layer, X, ws=ws), lambda: lib.gated(layer, X[:2], ws=ws),
                     lambda: lib.linear_backward(layer, X, dY, ws=ws),
                     lambda: lib.gated_backward(layer, X, dY, dH, ws=ws), lambda: lib.w4_linear(q4, X, ws=ws)):
            with pytest.raises(ValueError):
                call()
    assert lib.w4_linear(q4, X, ws=torch.zeros(1 << 20, dtype=torch.float32, device="cuda")).shape == (600, 256)
    lib.w4_sync_status(q4)
