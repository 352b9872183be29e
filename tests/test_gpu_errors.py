"""A call that the CUDA runtime refuses returns SLIM_ERR_CUDA, and only that
call does."""
import pytest
import torch

from gpu_util import to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


def test_a_refused_launch_leaves_the_next_call_alone(lib, tune):
    """Without the tensor-core path 16 x 65536 tokens are more token tiles than
    a grid's third dimension takes, so nothing is launched."""
    li = make_layer(LayerSpec("e", 128, 16, 0, 3, 0.02), 4)
    layer = lib.pack(to_dev(li.W))
    X = to_dev(li.X)
    want = lib.linear(layer, X)
    many = torch.zeros(16 * 65536, 128, dtype=torch.bfloat16, device="cuda")
    tune(SLIM_NO_PREFILL="1")
    for after in (lambda: lib.w4_unpack(lib.w4_pack(to_dev(li.W), 64)), lambda: lib.pack(to_dev(li.W)),
                  lambda: lib.unpack_dec(layer)):
        with pytest.raises(lib.SlimError) as e:
            lib.linear(layer, many)
        assert e.value.name == "SLIM_ERR_CUDA" and lib._lib.slim_last_cuda_error() != 0
        after()
    assert torch.equal(lib.linear(layer, X), want)
