"""Gated block on every tile of its tensor-core kernels, forced one by one: with
and without kept G and U, an adapter and a ragged rank, ragged token counts, and
more tiles than run at once.  Besides the norm over everything (operator_ref),
every block of 32 tokens x 32 columns is compared: it holds 1024 outputs, whose
error's share of their norm varies from block to block by much less than the
factor of 4 allowed, while a piece written to a wrong place is off by its whole
norm."""
from functools import lru_cache

import numpy as np
import pytest

import operator_ref as ref
from gpu_util import from_dev_bf16, to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu

TILES = ["2,64", "2,128", "2,192", "pair,128", "pair,192", "pair,224", "pair,240"]


@lru_cache(maxsize=4)
def case(K, F, r, M):
    lis = [make_layer(LayerSpec(f"t{i}", K, F, r, 3 + r + 31 * i, 0.02, max(1, K // 100), 20.0), M) for i in range(2)]
    G, U = ref.Linears(lis, r).forward(ref.f64(lis[0].X))
    return lis, G, U


def blocks_close(got, want):
    assert got.shape == want.shape and ref.rel(got, want) <= ref.FRO
    M, N = want.shape
    pad = [(0, -M % 32), (0, -N % 32)]
    err, val = (np.pad(a * a, pad).reshape(-(-M // 32), 32, -(-N // 32), 32).sum((1, 3)) for a in (got - want, want))
    assert (np.sqrt(err) <= 4 * ref.FRO * np.sqrt(val)).all()


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("r", [0, 20, 136])
@pytest.mark.parametrize("K,F,M", [(256, 2560, 2100), (384, 512, 257), (640, 256, 465)])
def test_gated_on_every_tile(lib, tune, K, F, M, r, tile):
    lis, G, U = case(K, F, r, M)
    layer = lib.pack_grouped([to_dev(li.W) for li in lis], [to_dev(li.L) for li in lis] if r else None,
                             [to_dev(li.R) for li in lis] if r else None)
    X = to_dev(lis[0].X)
    tune(SLIM_PREFILL_TILE=tile)
    name = "silu" if r else "gelu_tanh"
    H, GU = lib.gated(layer, X, act=name, keep=True)
    H2 = lib.gated(layer, X, act=name)
    lib.sync_status(layer)
    blocks_close(from_dev_bf16(H), ref.act(name, G) * U)
    blocks_close(from_dev_bf16(GU), np.concatenate([G, U], 1))
    assert (H == H2).all(), "keeping G and U changed H"


@pytest.mark.parametrize("tile", ["1,64", "1,128", "1,192", *TILES])
def test_a_forced_tile_serves_both_paths(lib, tune, tile):
    """A tile that one of the two paths lacks leaves that path its own choice."""
    lis, G, U = case(512, 512, 20, 300)
    layer = lib.pack_grouped(*([to_dev(getattr(li, k)) for li in lis] for k in "WLR"))
    X = to_dev(lis[0].X)
    tune(SLIM_PREFILL_TILE=tile)
    Y, H = lib.linear(layer, X), lib.gated(layer, X)
    lib.sync_status(layer)
    blocks_close(from_dev_bf16(Y), np.concatenate([G, U], 1))
    blocks_close(from_dev_bf16(H), ref.act("silu", G) * U)
