"""Activations and results in page-locked host memory, through the C interface: the same bits as on the device."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def pinned(t):
    return t.cpu().pin_memory()


def call(gq_lib, name, *args):
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    assert getattr(gq_lib.lib, name)(*args, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("t,code", [("q4_0", 2), ("q8_0", 8), ("q4_k", 12), ("mxfp4", 39)])
def test_grouped(gq_lib, cuda_dev, t, code):
    E, M, K, N, k = 5, 70, 512, 40, 2
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    W, U = (gq_lib.quantize(torch.randn((E * M, K), device=cuda_dev, generator=g) * 0.05, t) for _ in range(2))
    x = torch.randn((N, K), device=cuda_dev, generator=g)
    ids = torch.from_numpy(np.random.default_rng(2).integers(-1, E, (N, k)).astype(np.int32)).to(cuda_dev)
    offsets, pairs, places = gq_lib.moe_group(ids, E)
    R, before = N * k, torch.full((N * k, M), 3.0, device=cuda_dev)
    want = gq_lib.mul_mat_grouped(W, t, E, M, K, x, offsets, rows=pairs, top_k=k, out=before.clone())
    X, Y = pinned(x), pinned(before)
    call(gq_lib, "gq_mul_mat_grouped", W, code, E, M, K, X, N, pairs, k, offsets, R, Y)
    assert torch.equal(Y, want.cpu())
    h = gq_lib.mul_mat_grouped_swiglu(W, U, t, E, M, K, x, offsets, rows=pairs, top_k=k, out=before.clone())
    H = pinned(before)
    call(gq_lib, "gq_mul_mat_grouped_swiglu", W, U, code, E, M, K, X, N, pairs, k, offsets, R, H)
    assert torch.equal(H, h.cpu())
    w = torch.rand((N, k), device=cuda_dev, generator=g)
    y = gq_lib.moe_combine(want, places, w)
    Z = torch.zeros((N, M)).pin_memory()
    call(gq_lib, "gq_moe_combine", Y, R, M, places, w, N, k, Z)
    assert torch.equal(Z, y.cpu())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("r,K,M,N", [(16, 256, 70, 9), (64, 1024, 1024, 420), (16, 1024, 2048, 1100)])
def test_adapters(gq_lib, cuda_dev, dtype, r, K, M, N):
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    rand = lambda *s: torch.randn(s, device=cuda_dev, generator=g)
    adapters = gq_lib.LoraAdapters((rand(3, r, K) / 16).to(dtype), (rand(3, M, r) / 16).to(dtype))
    x, y0 = rand(N, K), rand(N, M)
    ids = torch.randint(-1, 3, (N,), device=cuda_dev, generator=g, dtype=torch.int32)
    want = gq_lib.lora_add(adapters, x, ids, y0).cpu()
    X, Y0, Y = pinned(x), pinned(y0), torch.zeros((N, M)).pin_memory()
    call(gq_lib, "gq_lora_add", ctypes.byref(adapters.c), X, N, ids, Y0, Y)
    assert torch.equal(Y, want)
    call(gq_lib, "gq_lora_add", ctypes.byref(adapters.c), X, N, ids, Y0, Y0)
    assert torch.equal(Y0, want)
