"""How the MXFP4 and expert calls behave among other calls: threads and streams at once, chains
with the older products, workspaces that grow, more tokens than one launch takes, values near
fp32's ends, misaligned arrays, empty ones, refusals of the binding."""
import threading

import numpy as np
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu


def matrix(M, K, seed, dev):
    W = (np.random.default_rng(seed).standard_normal((M, K)) * 0.05).astype(np.float32)
    blocks = ref.mx_pack(*ref.mx_quantize(W))
    return blocks, torch.from_numpy(blocks).to(dev)


def experts(gq_lib, dev, E, D, F, t="mxfp4"):
    g = torch.Generator(device=dev).manual_seed(E + D + F)
    parts = [gq_lib.quantize(torch.randn((r, k), device=dev, generator=g) * 0.05, t)
             for r, k in ((E * F, D), (E * F, D), (E * D, F))]
    return gq_lib.MoeExperts(*parts, t, E, D, F)


def moe_inputs(dev, E, D, N, k, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    ids = torch.stack([torch.randperm(E, device=dev, generator=g)[:k] for _ in range(N)]).to(torch.int32)
    return torch.randn((N, D), device=dev, generator=g), ids, torch.rand((N, k), device=dev, generator=g)


def calls(gq_lib, dev, seed):
    """Four calls on inputs of this seed, each with its result by itself."""
    M, K = 130, 544
    _, q = matrix(M, K, seed, dev)
    layer = experts(gq_lib, dev, 6, 64, 96)
    g = torch.Generator(device=dev).manual_seed(seed)
    xs = [torch.randn((n, K), device=dev, generator=g) for n in (1 + seed, 40)]
    m = moe_inputs(dev, 6, 64, 5 + seed, 2, seed)
    todo = [lambda: gq_lib.mul_mat(q, "mxfp4", M, K, xs[0]), lambda: gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, xs[0]),
            lambda: gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, xs[1]), lambda: gq_lib.moe_swiglu(layer, *m)]
    want = [f() for f in todo]
    torch.cuda.synchronize()
    return todo, want


@pytest.mark.parametrize("one_stream", [True, False])
def test_threads_at_once(gq_lib, cuda_dev, one_stream):
    work = [calls(gq_lib, cuda_dev, i) for i in range(4)]
    shared = torch.cuda.Stream()
    wrong = []

    def run(todo, want):
        with torch.cuda.stream(shared if one_stream else torch.cuda.Stream()):
            got = [[f() for f in todo] for _ in range(10)]
            torch.cuda.current_stream().synchronize()
            wrong.extend(1 for g in got for a, b in zip(g, want) if not torch.equal(a, b))

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and gq_lib.get_last_error() == 0


@pytest.mark.parametrize("N", [1, 2, 5, 40])
def test_chains_with_the_older_products(gq_lib, cuda_dev, N):
    """Each call's result is the next one's X, eagerly and in a graph; the same bits as with a
    synchronisation after every call."""
    D, F = 256, 512
    g = torch.Generator(device=cuda_dev).manual_seed(N)
    w = {t: (gq_lib.quantize(torch.randn((F, D), device=cuda_dev, generator=g) * 0.06, t),
             gq_lib.quantize(torch.randn((D, F), device=cuda_dev, generator=g) * 0.06, t))
         for t in ("q4_0", "q4_k", "mxfp4")}
    layer = experts(gq_lib, cuda_dev, 4, D, 64)
    x = torch.randn((N, D), device=cuda_dev, generator=g)
    ids = torch.randint(0, 4, (N, 2), device=cuda_dev, generator=g, dtype=torch.int32)
    wts = torch.rand((N, 2), device=cuda_dev, generator=g)
    sizes = [gq_lib.workspace_size(t, m, k, N) for t in w for m, k in ((F, D), (D, F))]
    n = max(sizes + [gq_lib.mx4x_workspace_size("mxfp4", D, F, N), layer.workspace_size(N, 2)])
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_dev)

    def step(wait):
        y = x
        for _ in range(3):
            for t in ("mxfp4", "q4_0", "mxfp4", "q4_k"):
                y = gq_lib.mul_mat_ws(w[t][0], t, F, D, y, ws)
                wait()
                y = gq_lib.mul_mat_ws(w[t][1], t, D, F, y, ws)
                wait()
                y = gq_lib.moe_swiglu(layer, y, ids, wts, workspace=ws) + x
                wait()
            y = gq_lib.mul_mat_mx4x(w["mxfp4"][0], "mxfp4", F, D, y, workspace=ws)
            wait()
            y = gq_lib.mul_mat_ws(w["q4_0"][1], "q4_0", D, F, y, ws)
            wait()
        return y

    want = step(torch.cuda.synchronize)
    assert torch.equal(step(lambda: None), want)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        y = step(lambda: None)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and gq_lib.get_last_error() == 0


def test_workspace_grows_between_calls(gq_lib, cuda_dev):
    M, K = 64, 96
    _, q = matrix(M, K, 1, cuda_dev)
    x = torch.randn((3000, K), device=cuda_dev)
    with torch.cuda.stream(torch.cuda.Stream()):   # a new stream: the library has no buffer yet
        first = gq_lib.mul_mat(q, "mxfp4", M, K, x[:1])
        big = gq_lib.mul_mat(q, "mxfp4", M, K, x)
        again = gq_lib.mul_mat(q, "mxfp4", M, K, x[:1])
        torch.cuda.current_stream().synchronize()
    # a token's sums do not depend on its neighbours' values, but their split over warps does on N
    want, tol = ref.product(*ref.weights("mxfp4", q.cpu().numpy(), M, K), x.cpu().numpy().astype(np.float64))
    assert torch.equal(first, again) and (np.abs(first.cpu().numpy() - want[:1]) <= tol[:1]).all()
    assert (np.abs(big.cpu().numpy() - want) <= tol).all()


def test_more_tokens_than_one_launch(gq_lib, cuda_dev):
    M, K, N = 40, 64, 8205
    blocks, q = matrix(M, K, 2, cuda_dev)
    x = torch.randn((N, K), device=cuda_dev)
    x64 = x.cpu().numpy().astype(np.float64)
    want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), x64)
    y = gq_lib.mul_mat(q, "mxfp4", M, K, x)
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
    z = gq_lib.mul_mat_noalloc(q, "mxfp4", M, K, x)
    assert (np.abs(z.cpu().numpy() - want) <= tol).all()
    y = gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x)
    want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), ref.mx_values(*ref.mx_quantize(x.cpu().numpy())))
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()


def test_rows_of_any_size(gq_lib, cuda_dev):
    """From subnormal activations to 2^100. Below 2^-110 the two terms keep an absolute 2^-149."""
    M, K = 40, 96
    blocks, q = matrix(M, K, 3, cuda_dev)
    x = np.random.default_rng(0).standard_normal((12, K)).astype(np.float32)
    scale = [0, 2.0 ** -140, 2.0 ** -126, 2.0 ** -112, 2.0 ** -108, 1e-20, 1e-3, 1, 1e5, 1e20, 2.0 ** 100, 1]
    x = (x.astype(np.float64) * np.array(scale)[:, None]).astype(np.float32)
    x[11, 1:] = 0
    w, z = ref.weights("mxfp4", blocks, M, K)
    want, tol = ref.product(w, z, x.astype(np.float64))
    tol = tol + 2.0 ** -148 * np.abs(w).sum(1) + 2.0 ** -148   # ... and the result's own rounding
    y = gq_lib.mul_mat(q, "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev)).cpu().numpy()
    assert (np.abs(y - want) <= tol).all() and (y[0] == 0).all()
    want, tol = ref.product(w, z, ref.mx_values(*ref.mx_quantize(x)))
    # few tokens: a subnormal sum per block; the tensor cores may lose a product below 2^-126
    for n, lost in ((12, 2.0 ** -148 * (K // 32 + 1)), (24, 2.0 ** -126 * K)):
        many = torch.from_numpy(np.concatenate([x] * (n // 12))).to(cuda_dev)
        y = gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, many).cpu().numpy()
        assert (np.abs(y[:12] - want) <= tol + lost).all() and (y[0] == 0).all()


def test_only_four_byte_aligned(gq_lib, cuda_dev):
    M, K = 70, 96
    _, q = matrix(M, K, 4, cuda_dev)
    layer = experts(gq_lib, cuda_dev, 3, 64, 32)

    def shifted(t, by):
        flat = torch.full((t.numel() + 8,), 9, dtype=t.dtype, device=cuda_dev)
        v = flat[by:by + t.numel()].view(t.shape)
        v.copy_(t)
        return flat, v

    for N in (1, 9, 30, 100):
        x = torch.randn((N, K), device=cuda_dev)
        m = moe_inputs(cuda_dev, 3, 64, N, 2)
        z = torch.randn((N, 37), device=cuda_dev)
        route = gq_lib.moe_route(z, 3)
        plain = [gq_lib.mul_mat(q, "mxfp4", M, K, x), gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x),
                 gq_lib.moe_swiglu(layer, *m)]
        for by in (1, 2, 3):
            xs = shifted(x, by)[1]
            ms = [shifted(t, by)[1] for t in m]
            outs = [shifted(t * 0, by) for t in plain]
            gq_lib.mul_mat(q, "mxfp4", M, K, xs, out=outs[0][1])
            gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, xs, out=outs[1][1])
            gq_lib.moe_swiglu(layer, *ms, out=outs[2][1])
            for (flat, got), want in zip(outs, plain):
                assert torch.equal(got, want)
                assert (flat[:by] == 9).all() and (flat[by + want.numel():] == 9).all()
            again = gq_lib.moe_route(shifted(z, by)[1], 3)
            assert torch.equal(again[0], route[0]) and torch.equal(again[1], route[1])


def test_empty_sizes(gq_lib, cuda_dev):
    _, q = matrix(4, 32, 5, cuda_dev)
    none = torch.empty(0, dtype=torch.uint8, device=cuda_dev)
    for f in (gq_lib.mul_mat, gq_lib.mul_mat_mx4x):
        assert f(q, "mxfp4", 4, 32, torch.empty((0, 32), device=cuda_dev)).shape == (0, 4)
        out = torch.full((3, 4), 7.0, device=cuda_dev)
        assert (f(none, "mxfp4", 4, 0, torch.empty((3, 0), device=cuda_dev), out=out) == 0).all()
        assert f(none, "mxfp4", 0, 32, torch.randn((3, 32), device=cuda_dev)).shape == (3, 0)
    assert gq_lib.moe_route(torch.empty((0, 8), device=cuda_dev), 2)[0].shape == (0, 2)
    layer = experts(gq_lib, cuda_dev, 2, 32, 32)
    x, ids, w = moe_inputs(cuda_dev, 2, 32, 3, 1)
    assert gq_lib.moe_swiglu(layer, x[:0], ids[:0], w[:0]).shape == (0, 32)


def test_binding_refuses(gq_lib, cuda_dev):
    M, K = 64, 64
    _, q = matrix(M, K, 6, cuda_dev)
    x = torch.randn((4, K), device=cuda_dev)
    layer = experts(gq_lib, cuda_dev, 3, 64, 32)
    xm, ids, w = moe_inputs(cuda_dev, 3, 64, 4, 2)
    wide = torch.randn((4, 2 * K), device=cuda_dev)[:, ::2]
    bad = [lambda: gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, wide), lambda: gq_lib.mul_mat(q, "mxfp4", M, K, wide),
           lambda: gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x.half()), lambda: gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x.t()),
           lambda: gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x, out=torch.empty((3, M), device=cuda_dev)),
           lambda: gq_lib.moe_route(wide, 2), lambda: gq_lib.moe_route(x.half(), 2),
           lambda: gq_lib.moe_swiglu(layer, wide[:, :64], ids, w), lambda: gq_lib.moe_swiglu(layer, xm, ids.long(), w),
           lambda: gq_lib.moe_swiglu(layer, xm, ids, w.double()), lambda: gq_lib.moe_swiglu(layer, xm, ids[:3], w[:3]),
           lambda: gq_lib.moe_swiglu(layer, xm, ids, w[:, :1]), lambda: gq_lib.moe_swiglu(layer, xm.cpu(), ids, w),
           lambda: gq_lib.moe_swiglu(layer, xm, ids, w, out=torch.empty((3, 64), device=cuda_dev))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: gq_lib.mul_mat_mx4x(q, "q4_0", M, K, x), lambda: gq_lib.moe_route(x, 65),
              lambda: gq_lib.moe_route(x, 0),
              lambda: gq_lib.moe_swiglu(layer, xm, ids, w, workspace=torch.empty(64, dtype=torch.uint8, device=cuda_dev))):
        with pytest.raises((ValueError, gq_lib.GQError)):
            f()
