"""MXFP4 and expert calls at the ends of what include/gq.h allows: arrays beyond 2^32 bytes, long
rows, the ends of the stated ranges, passes without work, graphs whose inputs change."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


def random_blocks(rows, K, nbytes, scale, dev, seed):
    """(rows, K / 32 * nbytes) of any codes under one scale (its bytes)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    b = torch.randint(0, 256, (rows * (K // 32), nbytes), device=dev, generator=g, dtype=torch.uint8)
    for i, v in enumerate(scale):
        b[:, i] = v
    return b.view(rows, -1)


MX_SCALE, Q4_SCALE = (122,), (0, 36)   # 2^-5; fp16 2^-6


def test_weights_beyond_32_bits(gq_lib, cuda_dev):
    """4.8 GB of blocks, 9e9 weights: rows at both ends and around every 2^31 and 2^32."""
    M, K = 1_100_003, 8192
    q = random_blocks(M, K, 17, MX_SCALE, cuda_dev, 0)
    row = q.shape[1]
    assert q.numel() > 2 ** 32
    at = [0, 1, 31, 32, M // 2, M - 33, M - 32, M - 2, M - 1]
    at += [n // row + i for n in (2 ** 31, 2 ** 32) for i in (-1, 0, 1)]
    at += [n // K + i for n in (2 ** 31, 2 ** 32, 2 ** 33) for i in (-1, 0, 1)]
    at = torch.tensor(sorted(set(at)), device=cuda_dev)
    w, z = ref.weights("mxfp4", q[at].cpu().numpy(), len(at), K)
    for N in (2, 20):
        x = torch.randn((N, K), device=cuda_dev)
        x64 = x.cpu().numpy()
        for f, xs in ((gq_lib.mul_mat, x64.astype(np.float64)),
                      (gq_lib.mul_mat_mx4x, ref.mx_values(*ref.mx_quantize(x64)))):
            want, tol = ref.product(w, z, xs)
            y = f(q, "mxfp4", M, K, x)[:, at].cpu().numpy()
            assert (np.abs(y - want) <= tol).all()
    rows = 530_000   # 4.3e9 weights, 17 GB
    W = gq_lib.dequantize(q[:rows], "mxfp4", rows, K)
    few = at[at < rows]
    assert np.array_equal(W[few].cpu().numpy(), w[:len(few)].astype(np.float32))
    last = torch.arange(rows - 3, rows, device=cuda_dev)
    want = ref.weights("mxfp4", q[last].cpu().numpy(), 3, K)[0]
    assert np.array_equal(W[last].cpu().numpy(), want.astype(np.float32))
    back = gq_lib.quantize(W, "mxfp4")
    assert torch.equal(gq_lib.dequantize(back[-3:], "mxfp4", 3, K), W[-3:])
    assert torch.equal(gq_lib.dequantize(back[few], "mxfp4", len(few), K), W[few])


def test_results_beyond_32_bits(gq_lib, cuda_dev):
    """1.08e9 results, 4.3 GB."""
    M, K, N = 1_048_583, 32, 1030
    q = random_blocks(M, K, 17, MX_SCALE, cuda_dev, 1)
    x = torch.randn((N, K), device=cuda_dev)
    x64 = x.cpu().numpy()
    at = torch.tensor([0, 5, M // 2, M - 2, M - 1], device=cuda_dev)
    w, z = ref.weights("mxfp4", q[at].cpu().numpy(), len(at), K)
    for f, xs in ((gq_lib.mul_mat, x64.astype(np.float64)),
                  (gq_lib.mul_mat_mx4x, ref.mx_values(*ref.mx_quantize(x64)))):
        want, tol = ref.product(w, z, xs)
        assert (np.abs(f(q, "mxfp4", M, K, x)[:, at].cpu().numpy() - want) <= tol).all()


def test_experts_beyond_32_bits(gq_lib, cuda_dev):
    """Three matrices of 4.8 GB, the first, middle and last experts at work."""
    E, D, F = 128, 2048, 32768
    mats = [random_blocks(r, k, 18, Q4_SCALE, cuda_dev, i) for i, (r, k) in
            enumerate(((E * F, D), (E * F, D), (E * D, F)))]
    assert all(m.numel() > 2 ** 32 for m in mats)
    layer = gq_lib.MoeExperts(*mats, "q4_0", E, D, F)
    ids = np.array([[0, 127], [127, 126], [63, 113], [114, 127]], np.int32)
    x = np.random.default_rng(0).standard_normal((4, D)).astype(np.float32) * np.float32(0.03)
    wts = np.random.default_rng(1).random((4, 2)).astype(np.float32)
    y = gq_lib.moe_swiglu(layer, *(torch.from_numpy(a).to(cuda_dev) for a in (x, ids, wts)))

    def values(m, rows, K, e):
        b = m[e * rows:(e + 1) * rows].view(rows, K // 32, 18)[:, :, 2:].long()
        return torch.cat([b & 15, b >> 4], 2).sub(8).double().mul(2.0 ** -6).view(rows, K)

    eps = ref.EPS
    for n in range(4):
        want = torch.zeros(D, dtype=torch.float64, device=cuda_dev)
        tol = torch.zeros_like(want)
        v = torch.from_numpy(x[n]).to(cuda_dev).double()
        for j in range(2):
            g, u = (values(m, F, D, ids[n, j]) for m in mats[:2])
            d = values(mats[2], D, F, ids[n, j])
            c, f = (D / 32 + 160) * eps, (F / 32 + 160) * eps
            a, b = g @ v, u @ v
            ea, eb = (c * (m.abs() @ v.abs()) + 2.0 ** -38 * v.abs().max() * m.abs().sum(1) for m in (g, u))
            s = a * torch.sigmoid(a)
            h = s * b
            eh = 1.1 * (b.abs() + eb) * ea + s.abs() * eb + 16 * eps * h.abs()
            w = float(wts[n, j])
            want += w * (d @ h)
            tol += w * (1.01 * f * (d.abs() @ h.abs()) + 2.0 ** -38 * h.abs().max() * d.abs().sum(1) +
                        d.abs() @ eh + 4 * eps * (d @ h).abs())
        assert ((y[n].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("K", [1 << 20, (1 << 21) + 32])
def test_long_rows(gq_lib, cuda_dev, K):
    """noalloc takes 8 or 7 of these tokens a pass."""
    M, N = 37, 17
    q = random_blocks(M, K, 17, MX_SCALE, cuda_dev, 2)
    x = torch.randn((N, K), device=cuda_dev)
    w = ref.weights("mxfp4", q.cpu().numpy(), M, K)
    x32 = x.cpu().numpy()
    want, tol = ref.product(*w, x32.astype(np.float64))
    for f in (gq_lib.mul_mat, gq_lib.mul_mat_noalloc):
        assert (np.abs(f(q, "mxfp4", M, K, x).cpu().numpy() - want) <= tol).all()
    want, tol = ref.product(*w, ref.mx_values(*ref.mx_quantize(x32)))
    for n in (3, N):
        y = gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x[:n]).cpu().numpy()
        assert (np.abs(y - want[:n]) <= tol[:n]).all()


def test_largest_weights(gq_lib, cuda_dev):
    """|What| just below 2^80, the border of the stated range, with small and large tokens."""
    M, K = 40, 96
    q = random_blocks(M, K, 17, (127 + 77,), cuda_dev, 3)
    x = np.random.default_rng(0).standard_normal((5, K)).astype(np.float32)
    x *= np.array([1, 1e-30, 1e10, 1e-38, 2.0 ** 30], np.float32)[:, None]
    w, z = ref.weights("mxfp4", q.cpu().numpy(), M, K)
    assert 2.0 ** 79 < np.abs(w).max() < 2.0 ** 80
    want, tol = ref.product(w, z, x.astype(np.float64))
    tol += 2.0 ** -148 * np.abs(w).sum(1)   # X below 2^-110
    y = gq_lib.mul_mat(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev)).cpu().numpy()
    assert (np.abs(y - want) <= tol).all()


@pytest.mark.parametrize("t", ("q4_0", "q8_0", "q4_k", "mxfp4"))
def test_small_hidden_vectors(gq_lib, cuda_dev, t):
    """Hidden values around and below 2^-110: what the bound has for them beside the usual terms."""
    layer = Layer(gq_lib, cuda_dev, t, 3, 256, 256)
    x, ids, w = layer.inputs(12, 2)
    x *= np.geomspace(1e-15, 1e-20, 12).astype(np.float32)[:, None]
    want, tol = ref.moe(*layer.ref, x.astype(np.float64), ids, w)
    for n in range(12):
        for j in range(2):
            a = np.abs(layer.ref[2][ids[n, j]][0]) + layer.ref[2][ids[n, j]][1]
            # the two terms' 2^-149 and h's own rounding (2^-150 where it is subnormal); per block
            # 2^-123; subnormal sums' roundings, 2^-150 each
            tol[n] += w[n, j] * (2.0 ** -147 * a.sum(1) + 2.0 ** -123 * (256 / 32)) + 2.0 ** -145
    y = layer.run(x, ids, w).cpu().numpy()
    assert (np.abs(y - want) <= tol).all()


def test_passes_without_work(gq_lib, cuda_dev):
    """700 tokens with two experts each are three passes; one of them has nobody at work."""
    layer = Layer(gq_lib, cuda_dev, "q4_0", 4, 64, 96)
    x, ids, w = layer.inputs(700, 2)
    ids[256:512] = -1
    y = layer.check(x, ids, w)
    assert (y[256:512] == 0).all()


def test_graph_with_changing_inputs(gq_lib, cuda_dev):
    """A captured router and layer follow what is in their inputs at each replay: other experts, all
    tokens on one, none, fewer."""
    E, D, F, N, k = 6, 96, 64, 24, 2
    layer = Layer(gq_lib, cuda_dev, "mxfp4", E, D, F)
    ws = torch.empty(layer.experts.workspace_size(N, k), dtype=torch.uint8, device=cuda_dev)
    x, ids, w = (torch.from_numpy(a).to(cuda_dev) for a in layer.inputs(N, k))
    out, graph = torch.zeros((N, D), device=cuda_dev), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gq_lib.moe_swiglu(layer.experts, x, ids, w, out=out, workspace=ws)
    for seed in range(5):
        a, b, c = layer.inputs(N, k, seed + 10)
        if seed == 1:
            b[:] = 3
        if seed == 2:
            b[:] = -1
        if seed == 3:
            b[5:] = E
        for dst, src in ((x, a), (ids, b), (w, c)):
            dst.copy_(torch.from_numpy(src))
        graph.replay()
        want, tol = ref.moe(*layer.ref, a.astype(np.float64), b, c)
        assert (np.abs(out.cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("N", [1, 20, 70])
def test_captured_batch(gq_lib, cuda_dev, N):
    """gq_mul_mat_batched_ws over MXFP4 matrices of several widths, which share one workspace."""
    shapes = [(100, 96), (64, 2048), (33, 544), (5, 32)]
    items = []
    for i, (M, K) in enumerate(shapes):
        q = random_blocks(M, K, 17, MX_SCALE, cuda_dev, 10 + i)
        items.append((q, M, K, torch.randn((N, K), device=cuda_dev), torch.zeros((N, M), device=cuda_dev)))
    problems = gq_lib.make_problems(items)
    size = gq_lib.batched_workspace_size(problems, "mxfp4", N)
    ws = torch.full((size + 256,), 90, dtype=torch.uint8, device=cuda_dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gq_lib.mul_mat_batched_ws(problems, "mxfp4", N, ws[:size])
        with pytest.raises(gq_lib.GQError):
            gq_lib.mul_mat_batched(problems, "mxfp4", N)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for q, M, K, x, y in items:
        assert torch.equal(y, gq_lib.mul_mat(q, "mxfp4", M, K, x))
    assert (ws[size:] == 90).all()


def test_fused_forms_with_more_tokens_than_one_pass(gq_lib, cuda_dev):
    M, K, N = 40, 64, 4100
    q, up = (random_blocks(M, K, 17, MX_SCALE, cuda_dev, s) for s in (20, 21))
    x = torch.randn((N, K), device=cuda_dev)
    x64 = x.cpu().numpy().astype(np.float64)
    w, z = ref.weights("mxfp4", q.cpu().numpy(), M, K)
    y, tol = ref.product(w, z, x64 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + 1e-5))
    got = gq_lib.mul_mat_rmsnorm(q, "mxfp4", M, K, x, torch.ones(K, device=cuda_dev), 1e-5)
    assert (np.abs(got.cpu().numpy() - y) <= 2 * tol).all()   # + the norm's own fp32 roundings
    g, eg = ref.product(w, z, x64)
    u, eu = ref.product(*ref.weights("mxfp4", up.cpu().numpy(), M, K), x64)
    s = g / (1 + np.exp(-g))
    got = gq_lib.mul_mat_swiglu(q, up, "mxfp4", M, K, x).cpu().numpy()
    assert (np.abs(got - s * u) <= 1.1 * (np.abs(u) + eu) * eg + np.abs(s) * eu + 16 * ref.EPS * np.abs(s * u)).all()
