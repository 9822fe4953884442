"""MXFP4 on the GPU: conversion bit-exact against the definition, mul_mat and the microscaled
product within the bounds that include/gq.h states."""
import numpy as np
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu


def special_rows(K):
    """Rows that decide between neighbours: ties, saturation, powers of two, zeros, tiny and
    huge blocks, negative zero, infinities and NaN."""
    rng = np.random.default_rng(5)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], np.float32)
    rows = [np.resize(np.concatenate([ties, -ties, np.nextafter(ties, 9, dtype=np.float32),
                                      np.nextafter(ties, 0, dtype=np.float32)]), K)]
    rows += [rows[0] * np.float32(2.0 ** s) for s in (-130, -126, -20, 3, 120, 125)]
    rows += [np.zeros(K, np.float32), np.full(K, -0.0, np.float32), np.full(K, 1e-45, np.float32),
             np.full(K, 2.0 ** -124, np.float32), np.full(K, 3.4028235e38, np.float32)]
    for bad in (np.inf, -np.inf, np.nan):
        r = rng.standard_normal(K).astype(np.float32)
        r[K // 2] = bad
        rows.append(r)
    rows += [rng.standard_normal(K).astype(np.float32) * np.float32(10.0 ** s) for s in (-38, -3, 0, 9)]
    return np.stack(rows)


@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (64, 32), (65, 2048), (300, 5632)])
def test_quantize_is_exact(gq_lib, cuda_dev, shape):
    W = np.random.default_rng(shape[0]).standard_normal(shape).astype(np.float32) * 0.02
    q = gq_lib.quantize(torch.from_numpy(W).to(cuda_dev), "mxfp4")
    codes, scales = ref.mx_quantize(W)
    assert np.array_equal(q.cpu().numpy(), ref.mx_pack(codes, scales))
    back = gq_lib.dequantize(q, "mxfp4", *shape).cpu().numpy()
    assert np.array_equal(back, ref.mx_values(codes, scales).astype(np.float32))


@pytest.mark.parametrize("offset", [0, 1])
def test_quantize_special_blocks(gq_lib, cuda_dev, offset):
    W = special_rows(128)
    flat = torch.empty(W.size + 4, device=cuda_dev)
    view = flat[offset:offset + W.size].view(W.shape)          # offset 1: only 4-byte aligned
    view.copy_(torch.from_numpy(W))
    q = gq_lib.quantize(view, "mxfp4")
    codes, scales = ref.mx_quantize(W)
    assert np.array_equal(q.cpu().numpy(), ref.mx_pack(codes, scales))
    out = torch.full((W.size + 8,), 7.0, device=cuda_dev)
    gq_lib.dequantize(q, "mxfp4", *W.shape, out=out[offset:offset + W.size].view(W.shape))
    got = out.cpu().numpy()
    assert np.array_equal(got[offset:offset + W.size].reshape(W.shape),
                          ref.mx_values(codes, scales).astype(np.float32), equal_nan=True)
    assert (got[:offset] == 7).all() and (got[offset + W.size:] == 7).all()


def test_dequantize_every_byte(gq_lib, cuda_dev):
    """Every scale byte with every code pair."""
    b = np.zeros((256, 17), np.uint8)
    b[:, 0] = np.arange(256)
    b[:, 1:] = np.random.default_rng(1).permutation(4096).reshape(256, 16).astype(np.uint8)
    back = gq_lib.dequantize(torch.from_numpy(b).to(cuda_dev), "mxfp4", 256, 32).cpu().numpy()
    assert np.array_equal(back, ref.mx_values(*ref.mx_unpack(b)).reshape(256, 32).astype(np.float32),
                          equal_nan=True)


def make(M, K, seed, dev):
    rng = np.random.default_rng(seed)
    W = (rng.standard_normal((M, K)) * 0.02 * np.exp(rng.standard_normal((M, 1)))).astype(np.float32)
    blocks = ref.mx_pack(*ref.mx_quantize(W))
    return blocks, torch.from_numpy(blocks).to(dev)


SHAPES = [(1, 32), (5, 64), (33, 96), (31, 1056), (130, 288), (256, 2048), (100, 2080), (2048, 544)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("N", [1, 3, 4, 5, 9, 16, 17, 40])
def test_mul_mat(gq_lib, cuda_dev, M, K, N):
    blocks, q = make(M, K, M + K, cuda_dev)
    x = np.random.default_rng(N).standard_normal((N, K)).astype(np.float32)
    x *= np.exp(2 * np.random.default_rng(N + 1).standard_normal((N, K))).astype(np.float32)
    y = gq_lib.mul_mat(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev))
    want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), x.astype(np.float64))
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
    assert torch.equal(y, gq_lib.mul_mat(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev)))


@pytest.mark.parametrize("M,K", SHAPES + [(129, 256), (300, 768)])
@pytest.mark.parametrize("N", [1, 7, 8, 9, 33, 64, 65, 130, 257, 520])
def test_mx4x(gq_lib, cuda_dev, M, K, N):
    blocks, q = make(M, K, M + K, cuda_dev)
    x = np.random.default_rng(N).standard_normal((N, K)).astype(np.float32)
    x *= np.exp(2 * np.random.default_rng(N + 1).standard_normal((N, 1))).astype(np.float32)
    y = gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev))
    want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), ref.mx_values(*ref.mx_quantize(x)))
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("N", [1, 5, 200])
def test_one_hot_returns_the_weights(gq_lib, cuda_dev, N):
    M, K = 96, 320
    blocks, q = make(M, K, 3, cuda_dev)
    w, _ = ref.weights("mxfp4", blocks, M, K)
    at = np.random.default_rng(N).integers(0, K, N)
    x = np.zeros((N, K), np.float32)
    x[np.arange(N), at] = 1.0
    for f in (gq_lib.mul_mat, gq_lib.mul_mat_mx4x):
        y = f(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev)).cpu().numpy()
        assert np.array_equal(y, w[:, at].T.astype(np.float32))


@pytest.mark.parametrize("N", [3, 130])
def test_bad_values_stay_in_their_rows(gq_lib, cuda_dev, N):
    """A NaN scale spoils its weight row, an infinity in X its token, and nothing else."""
    M, K = 100, 256
    blocks, _ = make(M, K, 9, cuda_dev)
    clean = ref.weights("mxfp4", blocks, M, K)
    blocks = blocks.copy()
    blocks.reshape(M, -1, 17)[41, 3, 0] = 255
    q = torch.from_numpy(blocks).to(cuda_dev)
    x = np.random.default_rng(N).standard_normal((N, K)).astype(np.float32)
    bad = x.copy()
    bad[1, 77], bad[2, 200] = np.inf, np.nan
    keep_n, keep_m = np.arange(N) != 1, np.arange(M) != 41
    keep_n &= np.arange(N) != 2
    for f, xs in ((gq_lib.mul_mat, x.astype(np.float64)),
                  (gq_lib.mul_mat_mx4x, ref.mx_values(*ref.mx_quantize(x)))):
        y = f(q, "mxfp4", M, K, torch.from_numpy(bad).to(cuda_dev)).cpu().numpy()
        want, tol = ref.product(*clean, xs)
        ok = np.ix_(keep_n, keep_m)
        assert (np.abs(y[ok] - want[ok]) <= tol[ok]).all()
        assert np.isnan(y[keep_n][:, 41]).all()
        assert not np.isfinite(y[1][keep_m]).any() and np.isnan(y[2][keep_m]).all()


@pytest.mark.parametrize("M,K,N", [(70, 96, 2), (64, 512, 20), (40, 544, 100)])
def test_every_entry_point(gq_lib, cuda_dev, M, K, N):
    """The forms with a caller's workspace, batched, without allocation and fused give the same
    products, and write nothing behind them."""
    blocks, q = make(M, K, 11, cuda_dev)
    x = torch.randn((N, K), device=cuda_dev)
    want = gq_lib.mul_mat(q, "mxfp4", M, K, x)
    n = gq_lib.workspace_size("mxfp4", M, K, N)
    ws = torch.full((n + 256,), 90, dtype=torch.uint8, device=cuda_dev)
    out = torch.full((N * M + 64,), 5.0, device=cuda_dev)
    gq_lib.mul_mat_ws(q, "mxfp4", M, K, x, ws[:n], out=out[:N * M].view(N, M))
    assert torch.equal(out[:N * M].view(N, M), want)
    assert (out[N * M:] == 5).all() and (ws[n:] == 90).all()
    assert torch.equal(gq_lib.mul_mat_noalloc(q, "mxfp4", M, K, x), want)
    ys = [torch.empty((N, M), device=cuda_dev) for _ in range(3)]
    gq_lib.mul_mat_batched([(q, M, K, x, ys[0]), (q, M, K, x * 2, ys[1]), (q, 0, K, x, ys[2])], "mxfp4", N)
    assert torch.equal(ys[0], want) and torch.equal(ys[1], want * 2)
    wx = gq_lib.mx4x_workspace_size("mxfp4", M, K, N)
    ws = torch.full((wx + 256,), 90, dtype=torch.uint8, device=cuda_dev)
    assert torch.equal(gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x, workspace=ws[:wx]),
                       gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x))
    assert (ws[wx:] == 90).all()
    w, z = ref.weights("mxfp4", blocks, M, K)
    x64 = x.cpu().numpy().astype(np.float64)
    xn = x64 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + 1e-5)
    y, tol = ref.product(w, z, xn)
    got = gq_lib.mul_mat_rmsnorm(q, "mxfp4", M, K, x, torch.ones(K, device=cuda_dev), 1e-5)
    assert (np.abs(got.cpu().numpy() - y) <= 2 * tol).all()   # + the norm's own fp32 roundings
    u, eu = ref.product(w, z, x64)
    s = u / (1 + np.exp(-u))
    got = gq_lib.mul_mat_swiglu(q, q, "mxfp4", M, K, x).cpu().numpy()
    assert (np.abs(got - s * u) <= 1.1 * (np.abs(u) + eu) * eu + np.abs(s) * eu + 1e-6 * np.abs(s * u)).all()


def test_weights_end_with_their_buffer(gq_lib, cuda_dev):
    """Sizes whose last row ends inside a 16-byte word of the weight buffer."""
    for M, K in ((1, 32), (3, 32), (7, 96), (33, 544)):
        blocks, _ = make(M, K, 1, cuda_dev)
        flat = torch.full((M * K // 32 * 17 + 64,), 255, dtype=torch.uint8, device=cuda_dev)
        flat[:blocks.size] = torch.from_numpy(blocks.reshape(-1)).to(cuda_dev)
        q = flat[:blocks.size].view(M, -1)
        x = np.random.default_rng(2).standard_normal((2, K)).astype(np.float32)
        want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), x.astype(np.float64))
        y = gq_lib.mul_mat(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev)).cpu().numpy()
        assert (np.abs(y - want) <= tol).all()


def test_pinned_host_activations(gq_lib, cuda_dev):
    M, K, N = 64, 96, 3
    _, q = make(M, K, 4, cuda_dev)
    x = torch.randn((N, K))
    for f in (gq_lib.mul_mat, gq_lib.mul_mat_mx4x):
        want = f(q, "mxfp4", M, K, x.to(cuda_dev)).cpu()
        got = f(q, "mxfp4", M, K, x.pin_memory())
        torch.cuda.synchronize()
        assert not got.is_cuda and torch.equal(got, want)


@pytest.mark.parametrize("N", [2, 200])
def test_captured_and_on_another_stream(gq_lib, cuda_dev, N):
    M, K = 96, 256
    _, q = make(M, K, 6, cuda_dev)
    x = torch.randn((N, K), device=cuda_dev)
    want = [f(q, "mxfp4", M, K, x) for f in (gq_lib.mul_mat, gq_lib.mul_mat_mx4x)]
    out = [torch.empty_like(w) for w in want]
    ws = [torch.empty(n, dtype=torch.uint8, device=cuda_dev) for n in
          (gq_lib.workspace_size("mxfp4", M, K, N), gq_lib.mx4x_workspace_size("mxfp4", M, K, N))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        gq_lib.mul_mat_ws(q, "mxfp4", M, K, x, ws[0], out=out[0])
        gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x, out=out[1], workspace=ws[1])
        for f in (gq_lib.mul_mat, gq_lib.mul_mat_mx4x):   # the library's workspace: refused
            with pytest.raises(gq_lib.GQError):
                f(q, "mxfp4", M, K, x, out=out[0])
    for o in out:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    with torch.cuda.stream(side):
        got = gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x)
    side.synchronize()
    assert torch.equal(got, want[1])
    assert gq_lib.get_last_error() == 0
