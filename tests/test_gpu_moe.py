"""The expert router and the mixture-of-experts layer against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu

TYPES = ("q4_0", "q8_0", "q4_k", "mxfp4")


# ---- router -------------------------------------------------------------------------------

def check_route(gq_lib, dev, z, k, renorm):
    ids, w = gq_lib.moe_route(torch.from_numpy(z).to(dev), k, renorm=renorm)
    want_ids, want_w = ref.route(z, k, renorm)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want_ids)
    # expf to 2 ulp, a sum of at most E terms, the division
    tol = (z.shape[1] + 8) * ref.EPS * want_w + 1e-44
    assert (np.abs(w.cpu().numpy() - want_w) <= tol).all()


@pytest.mark.parametrize("E", [1, 2, 31, 32, 33, 64, 100, 128, 255, 300, 512, 1000, 1024])
@pytest.mark.parametrize("N", [1, 5, 700])
def test_route(gq_lib, cuda_dev, E, N):
    z = (np.random.default_rng(E * N).standard_normal((N, E)) * 3).astype(np.float32)
    for k in sorted({1, min(E, 2), min(E, 8), min(E, 33), min(E, 64)}):
        check_route(gq_lib, cuda_dev, z, k, True)
        check_route(gq_lib, cuda_dev, z, k, False)


def test_route_ties_and_masks(gq_lib, cuda_dev):
    rng = np.random.default_rng(0)
    z = np.round(rng.standard_normal((400, 40)) * 2).astype(np.float32)      # many equal logits
    z[rng.random(z.shape) < 0.1] = -0.0
    z[rng.random(z.shape) < 0.3] = -np.inf
    z[rng.random(z.shape) < 0.05] = np.nan
    z[5], z[6], z[7] = -np.inf, np.nan, 0.0                                   # nothing, nothing, all equal
    z[8], z[9] = -3.4028235e38, 3.4028235e38                                  # the type's extremes
    z[10, 3] = z[10, 30] = np.inf
    z[11] = -np.inf
    z[11, 39] = -3.4028235e38                                                 # one expert left
    for k in (1, 3, 8, 40):
        check_route(gq_lib, cuda_dev, z, k, True)
        check_route(gq_lib, cuda_dev, z, k, False)
    ids, w = gq_lib.moe_route(torch.from_numpy(z).to(cuda_dev), 4)
    assert ids[5].tolist() == [0, 1, 2, 3] and w[5].tolist() == [0] * 4 and w[6].tolist() == [0] * 4


# ---- layer --------------------------------------------------------------------------------

def random_blocks(t, rows, K, rng):
    import oracle
    W = (rng.standard_normal((rows, K)) * 0.05).astype(np.float32)
    return ref.mx_pack(*ref.mx_quantize(W)) if t == "mxfp4" else oracle.quantize(t, W)


class Layer:
    def __init__(self, gq_lib, dev, t, E, D, F, seed=0, t_down=None):
        rng = np.random.default_rng(seed)
        t_down = t_down or t
        g, u = random_blocks(t, E * F, D, rng), random_blocks(t, E * F, D, rng)
        d = random_blocks(t_down, E * D, F, rng)
        cut = lambda tt, b, R, K: [tuple(a[e * R:(e + 1) * R] for a in ref.weights(tt, b, E * R, K))
                                   for e in range(E)]
        self.ref = (cut(t, g, F, D), cut(t, u, F, D), cut(t_down, d, D, F))
        up = lambda b: torch.from_numpy(np.ascontiguousarray(b)).to(dev)
        self.experts = gq_lib.MoeExperts(up(g), up(u), up(d), t, E, D, F, t_down=t_down)
        self.E, self.D, self.F, self.dev, self.lib = E, D, F, dev, gq_lib

    def inputs(self, N, k, seed=1):
        rng = np.random.default_rng(seed)
        x = (rng.standard_normal((N, self.D)) * np.exp(rng.standard_normal((N, 1)))).astype(np.float32)
        ids = rng.integers(0, self.E, (N, k)).astype(np.int32)
        w = rng.random((N, k)).astype(np.float32)
        return x, ids, w

    def run(self, x, ids, w, **kw):
        t = lambda a: torch.from_numpy(a).to(self.dev)
        return self.lib.moe_swiglu(self.experts, t(x), t(ids), t(w), **kw)

    def check(self, x, ids, w):
        y = self.run(x, ids, w)
        want, tol = ref.moe(*self.ref, x.astype(np.float64), ids, w)
        assert (np.abs(y.cpu().numpy() - want) <= tol).all()
        assert torch.equal(y, self.run(x, ids, w))        # the same bits every time
        return y


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("E,D,F,N,k", [(1, 256, 256, 1, 1), (4, 256, 512, 1, 2), (3, 512, 256, 5, 3),
                                       (8, 256, 256, 17, 4), (2, 256, 256, 40, 2), (5, 768, 256, 70, 8)])
def test_layer(gq_lib, cuda_dev, t, E, D, F, N, k):
    layer = Layer(gq_lib, cuda_dev, t, E, D, F)
    layer.check(*layer.inputs(N, k))


@pytest.mark.parametrize("t", ("q4_0", "q8_0", "mxfp4"))
@pytest.mark.parametrize("D,F", [(32, 32), (32, 96), (96, 32), (160, 352), (1056, 64), (64, 1376)])
def test_odd_widths(gq_lib, cuda_dev, t, D, F):
    layer = Layer(gq_lib, cuda_dev, t, 3, D, F)
    for N, k in ((1, 1), (6, 2), (33, 3)):
        layer.check(*layer.inputs(N, k))


def test_mixed_types(gq_lib, cuda_dev):
    for t, td in (("q4_0", "q8_0"), ("mxfp4", "q4_k"), ("q4_k", "mxfp4"), ("q8_0", "q4_0")):
        layer = Layer(gq_lib, cuda_dev, t, 3, 256, 256, t_down=td)
        layer.check(*layer.inputs(7, 2))


def test_every_token_on_one_expert(gq_lib, cuda_dev):
    layer = Layer(gq_lib, cuda_dev, "q4_0", 4, 64, 96)
    for N in (4, 5, 8, 9, 16, 17, 33, 100):
        x, ids, w = layer.inputs(N, 1)
        ids[:] = 2
        layer.check(x, ids, w)


def test_padding_duplicates_and_zero_weights(gq_lib, cuda_dev):
    layer = Layer(gq_lib, cuda_dev, "mxfp4", 5, 96, 64)
    x, ids, w = layer.inputs(12, 4)
    ids[0], ids[1], ids[2] = -1, 5, [3, 3, 3, 3]
    ids[3] = [-2147483648, 2147483647, 0, 4]
    w[4] = 0.0
    w[0] = np.nan                                  # weights of padding are not read into the sum
    y = layer.check(x, ids, np.where(np.isnan(w), 0, w).astype(np.float32))
    assert torch.equal(y, layer.run(x, ids, w))
    assert (y[0] == 0).all() and (y[1] == 0).all() and (y[4] == 0).all()
    ids[:] = -1                                    # nobody at work
    assert (layer.run(x, ids, w, out=torch.full((12, 96), 3.0, device=cuda_dev)) == 0).all()


def test_more_pairs_than_one_launch(gq_lib, cuda_dev):
    layer = Layer(gq_lib, cuda_dev, "q8_0", 6, 64, 64)
    for N, k in ((130, 6), (520, 1), (9, 64), (30, 33)):
        layer.check(*layer.inputs(N, k))


def test_many_experts(gq_lib, cuda_dev):
    layer = Layer(gq_lib, cuda_dev, "q4_0", 1024, 32, 32)
    layer.check(*layer.inputs(60, 8))
    x, ids, w = layer.inputs(1, 2)
    ids[:] = [[1023, 0]]
    layer.check(x, ids, w)


def test_values_of_any_size(gq_lib, cuda_dev):
    """Activations far from 1, zeros, and a token with an infinity: others keep their results."""
    layer = Layer(gq_lib, cuda_dev, "q4_0", 3, 128, 96)
    x, ids, w = layer.inputs(8, 2)
    x[1] *= 1e-12
    x[2] *= 1e6
    x[3] = 0
    x[4, 5:] = 0
    y = layer.check(x, ids, w)
    assert (y[3] == 0).all()
    x[6, 9] = np.inf
    z = layer.run(x, ids, w)
    keep = [n for n in range(8) if n != 6]
    assert torch.equal(z[keep], y[keep])


def test_router_then_layer(gq_lib, cuda_dev):
    """As they are used: RMS-normalised activations, router logits by mul_mat, route, layer; the
    residual of a second layer reads the first one's output."""
    E, D, F, N, k = 8, 256, 256, 6, 2
    layer = Layer(gq_lib, cuda_dev, "mxfp4", E, D, F)
    rng = np.random.default_rng(3)
    router = random_blocks("q8_0", E, D, rng)
    x = rng.standard_normal((N, D)).astype(np.float32)
    xs = torch.from_numpy(x).to(cuda_dev)
    logits = gq_lib.mul_mat(torch.from_numpy(router).to(cuda_dev), "q8_0", E, D, xs)
    ids, w = gq_lib.moe_route(logits, k)
    y = gq_lib.moe_swiglu(layer.experts, xs, ids, w)
    y2 = gq_lib.moe_swiglu(layer.experts, y, ids, w)
    want_ids, want_w = ref.route(logits.cpu().numpy(), k, True)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    want, tol = ref.moe(*layer.ref, x.astype(np.float64), want_ids, want_w)
    slack = 40 * ref.EPS * np.abs(want).max()      # the weights' own rounding
    assert (np.abs(y.cpu().numpy() - want) <= tol + slack).all()
    y64 = y.cpu().numpy().astype(np.float64)
    want2, tol2 = ref.moe(*layer.ref, y64, want_ids, want_w)
    assert (np.abs(y2.cpu().numpy() - want2) <= tol2 + 40 * ref.EPS * np.abs(want2).max()).all()


def test_workspace_capture_and_streams(gq_lib, cuda_dev):
    layer = Layer(gq_lib, cuda_dev, "q4_0", 4, 96, 64)
    x, ids, w = layer.inputs(20, 2)
    want = layer.run(x, ids, w)
    n = layer.experts.workspace_size(20, 2)
    ws = [torch.full((n + 256,), 90, dtype=torch.uint8, device=cuda_dev) for _ in range(2)]
    dev = [torch.from_numpy(a).to(cuda_dev) for a in (x, ids, w)]
    out = [torch.full((20 * 96 + 32,), 5.0, device=cuda_dev) for _ in range(2)]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            gq_lib.moe_swiglu(layer.experts, *dev, out=out[i][:20 * 96].view(20, 96), workspace=ws[i][:n])
            with pytest.raises(gq_lib.GQError):
                gq_lib.moe_swiglu(layer.experts, *dev, out=out[i][:20 * 96].view(20, 96))
        graphs.append(g)
    for _ in range(3):                             # two graphs at once, a workspace each
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i][:20 * 96].view(20, 96), want)
        assert (out[i][20 * 96:] == 5).all() and (ws[i][n:] == 90).all()
    assert gq_lib.get_last_error() == 0
