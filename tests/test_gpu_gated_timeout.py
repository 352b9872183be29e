"""When a wait of the gated block gives up, H and G, U are NaN (never values that
could pass for results), SLIM_ERR_TIMEOUT is reported, and the next call on the
same workspace is right."""
import pytest
import torch

from gpu_util import to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


def make(lib, K, F, r, M):
    lis = [make_layer(LayerSpec(f"o{i}", K, F, r, 5 + 31 * i, 0.02), M) for i in range(2)]
    layer = lib.pack_grouped([to_dev(li.W) for li in lis], [to_dev(li.L) for li in lis] if r else None,
                             [to_dev(li.R) for li in lis] if r else None)
    return layer, to_dev(lis[0].X)


def give_up(lib, layer, X, H, GU, ws, wait_us=500):
    rc = lib._lib.slim_test_gated_timeout(layer.ref, X.data_ptr(), X.shape[0], 0, H.data_ptr(),
                                          None if GU is None else GU.data_ptr(), ws.data_ptr(), ws.numel(), wait_us,
                                          torch.cuda.current_stream().cuda_stream)
    return lib.STATUS[rc]


@pytest.mark.parametrize("K,F,r,M,tile", [
    (512, 256, 16, 1, None), (512, 256, 0, 9, None), (640, 512, 20, 30, None),      # streamed
    (11008, 256, 16, 16, None), (14336, 256, 0, 16, None),                            # ... in panels
    (512, 256, 20, 300, "2,64"), (512, 512, 0, 300, "2,192"),
    (512, 256, 20, 300, "pair,128"), (512, 512, 0, 500, "pair,240"),
])
def test_gated_block_that_gives_up(lib, tune, K, F, r, M, tile):
    layer, X = make(lib, K, F, r, M)
    if tile:
        tune(SLIM_PREFILL_TILE=tile)
    ws = lib.gated_workspace(layer, M)
    want = lib.gated(layer, X, keep=True, ws=ws)
    H, GU = (torch.zeros_like(t) for t in want)
    assert give_up(lib, layer, X, H, GU, ws) == "SLIM_OK"
    with pytest.raises(lib.SlimError) as e:
        lib.sync_status(layer)
    assert e.value.name == "SLIM_ERR_TIMEOUT"
    assert H.isnan().all() and GU.isnan().all()
    H.zero_()
    assert give_up(lib, layer, X, H, None, ws) == "SLIM_OK"
    with pytest.raises(lib.SlimError):
        lib.sync_status(layer)
    assert H.isnan().all()
    assert all(torch.equal(a, b) for a, b in zip(lib.gated(layer, X, keep=True, ws=ws), want))
    lib.sync_status(layer)


def test_refusals(lib, tune):
    layer, X = make(lib, 256, 2560, 0, 2100)
    ws = lib.gated_workspace(layer, 2100)
    H = torch.zeros(2100, 2560, dtype=torch.bfloat16, device="cuda")
    assert give_up(lib, layer, X, H, None, ws, wait_us=0) == "SLIM_ERR_ARG"
    tune(SLIM_PREFILL_TILE="pair,128")       # 170 tiles: pairs would take several
    assert give_up(lib, layer, X, H, None, ws) == "SLIM_ERR_UNSUPPORTED"
    torch.cuda.synchronize()
    lib.sync_status(layer)
