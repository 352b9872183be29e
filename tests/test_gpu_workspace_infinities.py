"""What infinite and NaN gradients leave in a shared workspace is never taken for
the single-launch kernel's tagged words: a pair of bf16 whose second is +Inf (the
first any number, such as the launch count read as a subnormal) or a quiet NaN,
in every word behind the control block."""
import pytest
import torch

from gpu_util import to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu

K, F = 1024, 512


def make(lib, r, M, Fs=(F, F)):
    lis = [make_layer(LayerSpec(f"i{i}", K, n, r, 3 + i, 0.02), M) for i, n in enumerate(Fs)]
    return lib.pack_grouped(*([to_dev(getattr(li, k)) for li in lis] for k in "WLR")), to_dev(lis[0].X)


@pytest.mark.parametrize("M", [1, 16])
@pytest.mark.parametrize("second", [0x7F80, 0x7FC0, 0x7FFF])
def test_words_of_infinities(lib, M, second):
    layer, X = make(lib, 48, 16)
    assert layer.launches(M) == 1                       # the single-launch kernel
    X = X[:M]
    want = lib.linear(layer, X)
    ws = lib.workspace(layer, 16)
    for launch in range(6):
        assert int(ws[:4].view(torch.int32)) == launch
        words = ws[256:256 + (ws.numel() - 256) // 8 * 8].view(torch.int32).view(-1, 2)
        words[:, 0] = 0x3F800000                        # a plausible value: 1.0
        # every count the next launches could compare with, from this one's on
        words[:, 1] = (second << 16) + launch + 1 + torch.arange(words.shape[0], device="cuda", dtype=torch.int32) % 2
        assert torch.equal(lib.linear(layer, X, ws=ws), want)
    lib.sync_status(layer)


def test_backward_with_infinite_and_signalling_gradients(lib):
    """The workspace of passes over gradients of +Inf and of signalling NaN
    patterns (copied as they are for an odd number of rows) next serves the
    single-launch kernel."""
    layer, X = make(lib, 48, 200, (512, 301))
    want = lib.linear(layer, X[:3])
    ws = torch.zeros(max(layer.workspace_bytes(200), lib.backward_workspace(layer, 200).numel()), dtype=torch.uint8,
                     device="cuda")
    for bits in (0x7F80, 0x7F81, 0x7FA0):
        for launch in range(3):
            seq = int(ws[:4].view(torch.int32))
            dY = torch.empty(200, 813, dtype=torch.int32, device="cuda").fill_(bits).to(torch.int16)
            for i in range(3):
                dY[:, i::4] = seq + 1 + i % 2
            lib.linear_backward(layer, X, dY, ws=ws)
            assert torch.equal(lib.linear(layer, X[:3], ws=ws), want)
    lib.sync_status(layer)
