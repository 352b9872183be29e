"""Backward passes off the usual sizes: adapter gradients whose products run on
SM pairs, ranks of hundreds to thousands, 4-bit adapters, few tokens on layers
with many rows or many fused linears.

Tolerances: operator_ref.  A 4-bit adapter's factors are read as bf16(q s), one
rounding more than it counts for a product with them: n = 3 for dL and dR of the
linear (the factor, T or dT, the output), 4 for the gated block's (dG and dU
too), and sqrt(4) 2.26e-3 is still below FRO."""
import numpy as np
import pytest
import torch

import operator_ref as ref
import oracle
from gpu_util import from_dev_bf16, to_dev
from sparse_int4_linear_b200.workload import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


def members(K, Ns, r, M, seed):
    return [make_layer(LayerSpec(f"w{i}", K, n, r, seed + 31 * i, 0.02, max(1, K // 100), 20.0), M)
            for i, n in enumerate(Ns)]


def pack(lib, lis, r, **kw):
    return lib.pack_grouped([to_dev(li.W) for li in lis], [to_dev(li.L) for li in lis] if r else None,
                            [to_dev(li.R) for li in lis] if r else None, **kw)


def gradient(M, N, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * 0.01).bfloat16().cuda()


def linears(lis, r, bits=16):
    lin = ref.Linears(lis, r)
    if bits == 4:
        for i, li in enumerate(lis):
            qL, sL, qR, sR = oracle.quantize_adapters(li.L, li.R)
            lin.L[i], lin.R[i] = oracle.dequantize_adapter(qL, sL), oracle.dequantize_adapter(qR, sR)
    return lin


def split(d, Ns):
    return np.split(d, np.cumsum(Ns)[:-1], axis=1)


def check(got, want):
    for a, b, name in zip(got, want, ("dX", "dL", "dR")):
        assert (a is None) == (b is None), name
        if a is not None:
            assert tuple(a.shape) == b.shape
            assert ref.rel(from_dev_bf16(a), b) <= ref.FRO, name


@pytest.mark.parametrize("K,Ns,r,M", [
    (11008, (256, 256), 250, 40),        # dL [11008][2 x 250] on pairs, columns left out between the linears
    (11008, (512, 33), 256, 300),
    (128, (14336, 14336), 200, 40),      # dR [200][28672] on pairs, T's columns of the second linear from 208 on
    (256, (8192, 8192, 8201), 136, 130),
    (256, (256, 300), 300, 20),          # ranks beyond 256
    (384, (777,), 1000, 70),
    (128, (256, 256), 2048, 33),
    (256, (70,), 4096, 9),
    (128, (256,) * 7 + (5,), 500, 3),    # eight linears
    (512, (28672,), 16, 1),              # one token, two output tiles, a long sum
    (256, (28001,), 0, 1),
    (128, (20000,), 24, 5),
])
def test_linear_backward(lib, K, Ns, r, M):
    lis = members(K, Ns, r, M, 17 + K + r)
    layer = pack(lib, lis, r)
    X, dY = to_dev(lis[0].X), gradient(M, sum(Ns), M)
    got = lib.linear_backward(layer, X, dY)
    lib.sync_status(layer)
    check(got, linears(lis, r).backward(ref.f64(lis[0].X), split(from_dev_bf16(dY), Ns)))
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, lib.linear_backward(layer, X, dY)))


@pytest.mark.parametrize("K,Ns,r,M", [(1024, (512, 256), 20, 1), (640, (300,), 136, 64), (512, (256, 256, 256), 16, 300),
                                      (256, (8192, 8201), 200, 40)])
def test_linear_backward_with_4bit_adapters(lib, K, Ns, r, M):
    lis = members(K, Ns, r, M, 5 + K + r)
    layer = pack(lib, lis, r, adapter_bits=4)
    X, dY = to_dev(lis[0].X), gradient(M, sum(Ns), M)
    got = lib.linear_backward(layer, X, dY)
    lib.sync_status(layer)
    check(got, linears(lis, r, 4).backward(ref.f64(lis[0].X), split(from_dev_bf16(dY), Ns)))


@pytest.mark.parametrize("r,bits,M", [(300, 16, 20), (1000, 16, 100), (20, 4, 1), (136, 4, 300), (214, 4, 600)])
def test_gated_block_and_its_backward(lib, r, bits, M, K=384, F=512):
    lis = members(K, (F, F), r, M, 2 + r)
    layer = pack(lib, lis, r, adapter_bits=bits)
    lin = linears(lis, r, bits)
    x = ref.f64(lis[0].X)
    H, GU = lib.gated(layer, to_dev(lis[0].X), keep=True)
    G, U = lin.forward(x)
    assert ref.rel(from_dev_bf16(H), ref.act("silu", G) * U) <= ref.FRO
    dH = gradient(M, F, r)
    got = lib.gated_backward(layer, to_dev(lis[0].X), GU, dH)
    lib.sync_status(layer)
    G, U = split(from_dev_bf16(GU), (F, F))
    check(got, ref.gated_backward(lin, x, G, U, from_dev_bf16(dH), "silu"))
