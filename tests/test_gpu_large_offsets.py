"""Offsets beyond 2^31 elements: outputs of many tokens, and weights, that long.
Checked on samples of rows and columns against the same formulas in 64 bits."""
import numpy as np
import pytest
import torch

import operator_ref as ref

pytestmark = pytest.mark.gpu

M = 300_000


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def normal(g, *shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for i in range(0, shape[0], 1 << 16):
        n = min(1 << 16, shape[0] - i)
        out[i:i + n] = torch.randn((n, *shape[1:]), generator=g, device="cuda") * std
    return out


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def tokens():
    return torch.tensor([0, 1, 17, 131_071, 131_072, 262_143, 262_144, 299_000, M - 2, M - 1], device="cuda")


def weight(lib, layer, rows):
    q, s = lib.unpack_dec(layer)
    return q[rows].double() * s.view(torch.float16)[rows].double().repeat_interleave(128, 1)


def test_dense_4bit_many_outputs(lib, K=128, N=8200):
    g = torch.Generator(device="cuda").manual_seed(1)
    W, X = normal(g, N, K, std=0.02), normal(g, M, K)
    layer = lib.w4_pack(W, 64)
    Y = lib.w4_linear(layer, X)
    lib.w4_sync_status(layer)
    q, s = lib.w4_unpack(layer)
    t = tokens()
    assert rel(Y[t], X[t].double() @ (q.double() * s.view(torch.float16).double().repeat_interleave(64, 1)).T) <= ref.FRO


@pytest.mark.parametrize("tokens_", [1, 20, 600])
def test_dense_4bit_many_weights(lib, tokens_, K=65536, N=40000):
    g = torch.Generator(device="cuda").manual_seed(2)
    W, X = normal(g, N, K, std=0.02), normal(g, tokens_, K)
    layer = lib.w4_pack(W, 128)
    rows = torch.tensor([0, 15, 16, 32767, 32768, 32769, N - 1], device="cuda")
    qs = [ref.dense_w4(W[r:r + 1].view(torch.int16).cpu().numpy().view(np.uint16), 128)[2] for r in rows.tolist()]
    del W
    Y = lib.w4_linear(layer, X)
    lib.w4_sync_status(layer)
    assert rel(Y[:, rows], X.double() @ torch.from_numpy(np.concatenate(qs)).cuda().T) <= ref.FRO


def test_gated_block_and_backward_many_tokens(lib, K=128, F=4096, r=16):
    g = torch.Generator(device="cuda").manual_seed(3)
    W = [normal(g, F, K, std=0.02) for _ in range(2)]
    L = [normal(g, K, r, std=0.05) for _ in range(2)]
    R = [normal(g, r, F, std=0.05) for _ in range(2)]
    layer = lib.pack_grouped(W, L, R)
    X, t = normal(g, M, K), tokens()
    H, GU = lib.gated(layer, X, keep=True)
    lib.sync_status(layer)
    w = weight(lib, layer, slice(None))
    full = torch.cat([w[:F].T + L[0].double() @ R[0].double(), w[F:].T + L[1].double() @ R[1].double()], 1)
    gu = X[t].double() @ full
    assert rel(GU[t], gu) <= ref.FRO
    assert rel(H[t], torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) <= ref.FRO
    del H
    # a gradient that is not zero for the sampled tokens alone, so that dL and
    # dR are sums over them
    dH = torch.zeros(M, F, dtype=torch.bfloat16, device="cuda")
    dH[t] = normal(g, len(t), F, std=0.01)
    dX, dL, dR = lib.gated_backward(layer, X, GU, dH)
    lib.sync_status(layer)
    gu, dh = GU[t].double(), dH[t].double()
    s = torch.sigmoid(gu[:, :F])
    dy = torch.cat([dh * gu[:, F:] * (s + gu[:, :F] * s * (1 - s)), dh * gu[:, :F] * s], 1)
    assert rel(dX[t], dy @ full.T) <= ref.FRO
    dX[t] = 0
    assert not dX.any()
    dT = [dy[:, i * F:(i + 1) * F] @ R[i].double().T for i in range(2)]
    assert rel(dL, torch.cat([X[t].double().T @ d for d in dT], 1)) <= ref.FRO
    assert rel(dR, torch.cat([(X[t].double() @ L[i].double()).T @ dy[:, i * F:(i + 1) * F] for i in range(2)], 1)) <= ref.FRO


def test_linear_backward_many_weights(lib, K=65536, N=40000, tokens_=24):
    g = torch.Generator(device="cuda").manual_seed(4)
    W = normal(g, N, K, std=0.02)
    layer = lib.pack(W)
    del W
    rows = torch.tensor([0, 15, 16, 32767, 32768, 32769, N - 1], device="cuda")
    w = weight(lib, layer, rows)
    for m in (tokens_, 600):        # expanded inside the product, and in memory
        dY = torch.zeros(m, N, dtype=torch.bfloat16, device="cuda")
        dY[:, rows] = normal(g, m, len(rows))
        dX = lib.linear_backward(layer, None, dY, need=("dX",))[0]
        lib.sync_status(layer)
        assert rel(dX, dY[:, rows].double() @ w) <= ref.FRO
