"""How the dense 4-bit linear's kernel for few tokens splits its work, from the
library's own planner (host only): every rank of a cluster has a chunk of every
panel, whatever the row length the format accepts (K up to 2^20)."""
import ctypes

import pytest
import torch

from sparse_int4_linear_b200 import slim

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder buffers: host-only checks run where no GPU is visible")

P = 1 << 30          # placeholder device address (never touched)
lib = slim._lib


def plan(K, N, group, M):
    L = slim.SlimW4Desc()
    rc = lib.slim_w4_init(ctypes.byref(L), K, N, group, P, lib.slim_w4_bytes(K, N, group), None)
    assert rc in (0, -7) and L.magic
    out = (ctypes.c_int32 * 4)()
    assert lib.slim_w4_plan(ctypes.byref(L), M, out) == 0
    return list(out)


def check(K, N, group, M):
    S, panels, ckp, ctas = plan(K, N, group, M)
    assert S >= 1 and panels >= 1 and 1 <= ctas <= -(-N // 16)
    C = K // 128
    shares = {(r + 1) * C // S - r * C // S for r in range(S)}
    for n in shares:
        # panels of ckp chunks, the last one with 1 to ckp
        assert (panels - 1) * ckp < n <= panels * ckp, (K, N, group, M, S, panels, ckp, n)


@pytest.mark.parametrize("N", [1, 16, 300, 592, 1000, 1024, 1184, 4096])
def test_every_rank_has_a_chunk_of_every_panel(N):
    for i, C in enumerate(range(1, (1 << 20) // 128 + 1)):
        check(C * 128, N, (32, 64, 128)[i % 3], (16, 1, 8, 9, 15)[i % 5])


@pytest.mark.parametrize("K,N,group,M", [(238208, 1000, 32, 16), (254080, 1024, 128, 16), (1015936, 16, 128, 8),
                                         (1 << 20, 16, 32, 16)])
def test_uneven_ranks_of_long_rows(K, N, group, M):
    check(K, N, group, M)


def test_plan_refusals_and_other_paths():
    L = slim.SlimW4Desc()
    out = (ctypes.c_int32 * 4)()
    assert slim.STATUS[lib.slim_w4_plan(ctypes.byref(L), 1, out)] == "SLIM_ERR_STATE"
    assert plan(4096, 4096, 128, 0) == [0] * 4 and plan(4096, 4096, 128, 2000) == [0] * 4
    assert plan(4096, 4096, 128, 16)[0] >= 1
