"""Grouped products and adapters at the far ends of K and M."""
import numpy as np
import pytest
import torch

import grouped_reference as gr
from test_gpu_grouped import Experts, near, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,K", [("q4_0", 1 << 20), ("q8_0", (1 << 20) + 32), ("q4_k", 1 << 20), ("mxfp4", (1 << 20) + 96)])
def test_long_rows(gq_lib, cuda_dev, t, K):
    x = Experts(gq_lib, cuda_dev, t, 1, 5, K)
    for n in (3, 40, 130):
        x.check(tokens(n, K), [0, n])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,r,K,M", [(1, 8, 1 << 24, 40), (2, 8, 1 << 21, 64), (1, 8, 32, 1 << 23), (3, 8, 64, 1 << 20),
                                     (20, 256, 4096, 1 << 18)])
def test_adapters(gq_lib, cuda_dev, dtype, N, r, K, M):
    """The largest K and M, by tiles and by single tokens."""
    g = torch.Generator(device=cuda_dev).manual_seed(K + M)
    rand = lambda *s: torch.randn(s, device=cuda_dev, generator=g)
    A, B = (rand(2, r, K) / K ** 0.5).to(dtype), (rand(2, M, r) * 0.1).to(dtype)
    X, Y = rand(N, K), rand(N, M)
    ids = torch.arange(N, device=cuda_dev, dtype=torch.int32) % 2
    got = gq_lib.lora_add(gq_lib.LoraAdapters(A, B), X, ids, Y)
    for n in range(0, N, 7):
        a, b, x = A[n % 2].double(), B[n % 2].double(), X[n].double()
        want = Y[n].double() + b @ (a @ x)
        down = (K / 32 + r / 32 + 400) * 2.0 ** -24 * (a.abs() @ x.abs()) + 2.0 ** -38 * x.abs().max() * a.abs().sum(1)
        tol = 2.0 ** -23 * Y[n].double().abs() + b.abs() @ down + 2.0 ** -38 * (a @ x).abs().max() * b.abs().sum(1)
        assert bool(((got[n].double() - want).abs() <= tol).all())


def test_one_weight_row(gq_lib, cuda_dev):
    """M = 1: one row of a tile of 128, many experts and units."""
    for t in ("q4_0", "q8_0", "q4_k", "mxfp4"):
        x = Experts(gq_lib, cuda_dev, t, 900, 1, 256)
        n = np.random.default_rng(3).integers(0, 5, 900)
        x.check(tokens(n.sum(), 256), np.concatenate([[0], np.cumsum(n)]))
