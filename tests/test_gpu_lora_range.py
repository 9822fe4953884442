"""Adapters whose entries are among fp16's subnormals, and activations at the end of fp32's range, in tiles of
tokens and by single tokens."""
import numpy as np
import pytest
import torch

import grouped_reference as gr

pytestmark = pytest.mark.gpu

# N above N * r * (K + M) = 5e7: tiles (every form of the kernels); below: a few tokens.
SHAPES = [(16, 1024, 2048, 1100), (16, 1056, 2050, 1030), (8, 544, 2600, 2003), (32, 1568, 1024, 700),
          (64, 1024, 1024, 420), (40, 800, 1100, 700), (64, 992, 1058, 401), (128, 1024, 1056, 200),
          (136, 1024, 770, 230), (16, 1024, 2048, 7)]
L = 3


def entries(rng, shape, exponent):
    """fp16 values of up to 2^exponent; below 2^-14 multiples of 2^-24."""
    return (rng.standard_normal(shape) * 2.0 ** exponent / 3).astype(np.float16)


def floor(a):
    """What an entry counts in the bound: fp16's subnormals as 2^-14."""
    f = np.abs(a).astype(np.float64)
    return np.where(f > 0, np.maximum(f, 2.0 ** -14), 0) if a.dtype == np.float16 else f


def check(gq_lib, dev, A, B, x, y0=None, tiles=True):
    L, r, K = A.shape
    N, M = len(x), B.shape[1]
    ids = (np.arange(N) * 7 % L).astype(np.int32)
    y0 = np.zeros((N, M), np.float32) if y0 is None else y0
    up = lambda a: torch.from_numpy(a).to(dev)
    got = gq_lib.lora_add(gq_lib.LoraAdapters(up(A) if A.dtype == np.float16 else up(A).bfloat16(),
                                              up(B) if B.dtype == np.float16 else up(B).bfloat16()),
                          up(x), up(ids), up(y0)).cpu().double().numpy()
    f = lambda a: a.astype(np.float64)
    want, tol = gr.lora(f(A), f(B), np.ones(L), f(x), ids, f(y0))
    if tiles:
        tol = gr.lora(floor(A), floor(B), np.ones(L), np.abs(f(x)), ids, f(y0))[1]
    err = np.abs(got - want)
    assert np.isfinite(got).all() and (err <= tol).all(), f"{(err / np.maximum(tol, 1e-300)).max()} of the bound"


@pytest.mark.parametrize("r,K,M,N", SHAPES)
@pytest.mark.parametrize("a,b", [(-15, 0), (-21, 0), (0, -15), (0, -21), (-18, -18)])
def test_subnormal_entries(gq_lib, cuda_dev, r, K, M, N, a, b):
    """The whole of A or of B below 2^-14. By single tokens they are as near as larger ones; in tiles they count as
    2^-14, for the tensor cores align products by nominal exponents."""
    rng = np.random.default_rng(r + N)
    check(gq_lib, cuda_dev, entries(rng, (L, r, K), a), entries(rng, (L, M, r), b),
          rng.standard_normal((N, K)).astype(np.float32), tiles=N * r * (K + M) > 50000000)


@pytest.mark.parametrize("r,K,M,N", SHAPES)
@pytest.mark.parametrize("which", ["A", "B", "both"])
def test_subnormal_entries_beside_large_ones(gq_lib, cuda_dev, r, K, M, N, which):
    """Entries of 2 and more, up to the largest, stand among them; their x (their r numbers) are zeros."""
    rng = np.random.default_rng(r + N)
    A, B = entries(rng, (L, r, K), -17), entries(rng, (L, M, r), -17)
    x = rng.standard_normal((N, K)).astype(np.float32)
    if which != "B":
        A[:, :, ::32] = rng.choice(np.array([2, -3.5, 65504, 1000], np.float16), A[:, :, ::32].shape)
        x[:, ::32] = 0
        A[0, :, ::32], x[::7, 32] = 0, 1.0            # an adapter without; and tokens that use them
    if which != "A":
        B[:, :, ::8] = rng.choice(np.array([2, -3.5, 65504, 1000], np.float16), B[:, :, ::8].shape)
        A[:, ::8] = 0
    check(gq_lib, cuda_dev, A, B, x)


@pytest.mark.parametrize("r,K,M,N", SHAPES)
@pytest.mark.parametrize("f16", [True, False])
def test_largest_activations(gq_lib, cuda_dev, r, K, M, N, f16):
    """The last floats before infinity: no term of theirs is one."""
    rng = np.random.default_rng(r + N)
    A, B = np.zeros((L, r, K), np.float32), (rng.integers(-8, 9, (L, M, r)) / 8).astype(np.float32)
    x = rng.standard_normal((N, K)).astype(np.float32)
    x[:, 40] = np.float32(3.4028234e38) * rng.choice([-1, 1], N)
    x[::2, 40] = np.float32(3.397e38)
    A[:, :, 40] = rng.integers(-4, 5, (L, r)) * 2.0 ** -12
    A[:, :, 3] = 0.5
    y0 = rng.standard_normal((N, M)).astype(np.float32)
    if f16:
        A, B = A.astype(np.float16), B.astype(np.float16)
    check(gq_lib, cuda_dev, A, B, x, y0)
