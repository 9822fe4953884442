"""Every form of the MXFP4 kernels that large shapes take: the microscaled product's tile widths,
several tiles a CTA and both ways of laying operands out; several units a warp in the few-token
kernel, dense and over experts; the quantizer's four blocks a thread. And how far all are off in
the mean, beside the worst-case bounds of the other tests."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu

SMS = 152


def ceil(a, b):
    return -(-a // b)


def tile_width(gq_lib, M, K, N):
    """Columns of the product's tiles, from the workspace: records of 128 weight rows and of as many
    token rows, 128 bytes a row and 512 for each 128 rows' scales of four blocks, twice."""
    record = lambda rows: rows * 128 + 2 * ceil(rows, 128) * 512
    k = ceil(K, 256)
    x = gq_lib.mx4x_workspace_size("mxfp4", M, K, N) - ceil(M, 128) * k * record(128)
    width = [bn for bn in (64, 128, 192) if ceil(N, bn) * k * record(bn) == x]
    assert len(width) == 1
    return width[0]


def four_blocks_a_thread(M, K, N, bn):
    k = ceil(K, 256)
    return ceil(M, 128) * k + ceil(N, bn) * k * (bn // 32) >= 4 * SMS


# M, K, N, columns of a tile, rounds of tiles over the SMs, four blocks a thread in the preparation
PRODUCTS = [(5601, 544, 500, 192, 1, False),
            (5601, 4000, 500, 192, 1, True),
            (9000, 96, 1003, 192, 3, False),
            (11000, 64, 3000, 192, 10, False),
            (2040, 288, 2039, 128, 2, False),
            (2000, 2080, 2000, 128, 2, True),
            (3001, 2080, 385, 128, 1, False),
            (20000, 2080, 40, 64, 2, True),
            (80000, 64, 20, 64, 5, True)]


def weights(M, K, seed):
    """Blocks of any codes under scales of 2^-11 to 2^-4."""
    rng = np.random.default_rng(seed)
    b = rng.integers(0, 256, (M, K // 32, 17), np.uint8)
    b[:, :, 0] = rng.integers(116, 124, (M, K // 32), np.uint8)
    return b.reshape(M, -1)


@pytest.mark.parametrize("M,K,N,bn,rounds,four", PRODUCTS)
def test_microscaled_product(gq_lib, cuda_dev, M, K, N, bn, rounds, four):
    assert tile_width(gq_lib, M, K, N) == bn and four_blocks_a_thread(M, K, N, bn) == four
    assert ceil(ceil(M, 128) * ceil(N, bn), SMS) == rounds
    blocks = weights(M, K, M)
    x = np.random.default_rng(N).standard_normal((N, K), np.float32)
    x *= np.exp(2 * np.random.default_rng(1).standard_normal((N, 1))).astype(np.float32)
    q, xs = torch.from_numpy(blocks).to(cuda_dev), torch.from_numpy(x).to(cuda_dev)
    size = gq_lib.mx4x_workspace_size("mxfp4", M, K, N)
    ws = torch.full((size + 256,), 90, dtype=torch.uint8, device=cuda_dev)
    out = torch.full((N * M + 64,), 5.0, device=cuda_dev)
    gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, xs, out=out[:N * M].view(N, M), workspace=ws[:size])
    y = out[:N * M].view(N, M)
    want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), ref.mx_values(*ref.mx_quantize(x)))
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
    assert (out[N * M:] == 5).all() and (ws[size:] == 90).all()
    shifted = torch.empty(N * K + 1, device=cuda_dev)[1:].view(N, K).copy_(xs)   # 4-byte aligned X
    assert torch.equal(gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, shifted), y)
    assert gq_lib.get_last_error() == 0


@pytest.mark.parametrize("M,K,N", [(5601, 544, 500), (9000, 96, 1003), (2040, 288, 2039)])
def test_bad_values_stay_in_their_rows(gq_lib, cuda_dev, M, K, N):
    """In wide tiles, with tokens beyond the first 128 of a tile and in a later tile."""
    blocks = weights(M, K, 2).copy()
    rows, tokens = np.array([3, M // 2, M - 1]), np.array([1, 130, 191, 193, N - 1])
    x = np.random.default_rng(N).standard_normal((N, K), np.float32)
    clean = torch.from_numpy(x).to(cuda_dev)
    want = gq_lib.mul_mat_mx4x(torch.from_numpy(blocks).to(cuda_dev), "mxfp4", M, K, clean)
    blocks.reshape(M, -1, 17)[rows, 1, 0] = 255
    x[tokens[::2], K // 2], x[tokens[1::2], K - 1] = np.inf, np.nan
    y = gq_lib.mul_mat_mx4x(torch.from_numpy(blocks).to(cuda_dev), "mxfp4", M, K,
                            torch.from_numpy(x).to(cuda_dev))
    bad = torch.zeros((N, M), dtype=torch.bool, device=cuda_dev)
    bad[torch.from_numpy(tokens).to(cuda_dev)] = True
    bad[:, torch.from_numpy(rows).to(cuda_dev)] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("M,K,N", [(5601, 544, 500), (9000, 96, 1003), (2040, 288, 2039), (80000, 64, 20)])
def test_one_hot_returns_the_weights(gq_lib, cuda_dev, M, K, N):
    blocks = weights(M, K, 3)
    w, _ = ref.weights("mxfp4", blocks, M, K)
    at = np.random.default_rng(N).integers(0, K, N)
    x = np.zeros((N, K), np.float32)
    x[np.arange(N), at] = 1.0
    y = gq_lib.mul_mat_mx4x(torch.from_numpy(blocks).to(cuda_dev), "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev))
    assert np.array_equal(y.cpu().numpy(), w[:, at].T.astype(np.float32))


def test_products_follow_each_other(gq_lib, cuda_dev):
    """One workspace, tiles of every width in turn: each result the one by itself."""
    shapes = [s[:3] for s in PRODUCTS]
    size = max(gq_lib.mx4x_workspace_size("mxfp4", *s) for s in shapes)
    ws = torch.empty(size, dtype=torch.uint8, device=cuda_dev)
    todo = []
    for M, K, N in shapes:
        q = gq_lib.quantize(torch.randn((M, K), device=cuda_dev), "mxfp4")
        x = torch.randn((N, K), device=cuda_dev)
        todo.append((q, M, K, x, gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x)))
    torch.cuda.synchronize()
    for _ in range(3):
        got = [gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, x, workspace=ws) for q, M, K, x, _ in todo]
        assert all(torch.equal(y, t[4]) for y, t in zip(got, todo))
    assert gq_lib.get_last_error() == 0


# More units (32 rows, 8 or 16 tokens) than row warps: runs of units that cross from one group of
# tokens to the next, without and with a split of K over warps.
@pytest.mark.parametrize("M,K,N", [(80011, 96, 8), (80011, 544, 5), (33001, 96, 40), (33001, 544, 40), (9000, 288, 131)])
def test_several_units_a_warp(gq_lib, cuda_dev, M, K, N):
    blocks = weights(M, K, K)
    x = np.random.default_rng(N).standard_normal((N, K), np.float32)
    x *= np.exp(2 * np.random.default_rng(1).standard_normal((N, 1))).astype(np.float32)
    q, xs = torch.from_numpy(blocks).to(cuda_dev), torch.from_numpy(x).to(cuda_dev)
    units = ceil(M, 32) * (ceil(N, 16) if N > 8 else 1)
    assert units > SMS * 16   # at most, with no split of K
    w = ref.weights("mxfp4", blocks, M, K)
    want, tol = ref.product(*w, x.astype(np.float64))
    y = gq_lib.mul_mat(q, "mxfp4", M, K, xs)
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
    assert torch.equal(y, gq_lib.mul_mat(q, "mxfp4", M, K, xs))
    if N <= 16:
        y = gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, xs)
        want, tol = ref.product(*w, ref.mx_values(*ref.mx_quantize(x)))
        assert (np.abs(y.cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("t", ("q4_0", "q8_0", "q4_k", "mxfp4"))
@pytest.mark.parametrize("wide", [False, True])
def test_several_units_a_warp_over_experts(gq_lib, cuda_dev, t, wide):
    """Widths in turn, so that gate/up has the many units once, and down once."""
    unit = 256 if t == "q4_k" else 32
    for D, F in ((unit, 2048), (2048, unit)):
        E, N, k = (40, 64, 8) if wide else (48, 50, 8)   # 12.8 and 8.3 tokens an expert
        layer = Layer(gq_lib, cuda_dev, t, E, D, F)
        assert max(D, F) // 32 * E > SMS * 16
        x, ids, w = layer.inputs(N, k)
        y = layer.run(x, ids, w)
        some = np.arange(0, N, 5)   # tokens; their pairs lie anywhere in the experts' groups
        want, tol = ref.moe(*layer.ref, x[some].astype(np.float64), ids[some], w[some])
        assert (np.abs(y.cpu().numpy()[some] - want) <= tol).all()
        assert torch.equal(y, layer.run(x, ids, w))


@pytest.mark.parametrize("offset", [0, 1])
def test_four_blocks_a_thread(gq_lib, cuda_dev, offset):
    """From 38912 blocks, with a last step that is not full, and fp32 arrays only 4-byte aligned."""
    M, K = 40003, 32
    W = np.random.default_rng(7).standard_normal((M, K), np.float32)
    W[5], W[M - 1, 3], W[M // 2] = 0, np.inf, 2.0 ** -126
    flat = torch.empty(W.size + 8, device=cuda_dev)
    view = flat[offset:offset + W.size].view(M, K)
    view.copy_(torch.from_numpy(W))
    blocks = torch.full((M * 17 + 64,), 90, dtype=torch.uint8, device=cuda_dev)
    gq_lib.quantize(view, "mxfp4", out=blocks[:M * 17].view(M, 17))
    codes, scales = ref.mx_quantize(W)
    assert np.array_equal(blocks[:M * 17].view(M, 17).cpu().numpy(), ref.mx_pack(codes, scales))
    assert (blocks[M * 17:] == 90).all()
    out = torch.full((W.size + 8,), 7.0, device=cuda_dev)
    gq_lib.dequantize(blocks[:M * 17].view(M, 17), "mxfp4", M, K, out=out[offset:offset + W.size].view(M, K))
    got = out.cpu().numpy()
    assert np.array_equal(got[offset:offset + W.size].reshape(M, K), ref.mx_values(codes, scales).astype(np.float32),
                          equal_nan=True)
    assert (got[:offset] == 7).all() and (got[offset + W.size:] == 7).all()


# Root mean square error over the results' root mean square, on random data at ordinary sizes. The
# documented errors are 2e-7 to 5e-7; twice the larger is the limit. Losing the small term of X
# would make it 2^-13 or so, losing five of its eleven bits 1e-6.
LIMIT = 1e-6


def off(y, want):
    return np.sqrt(((y.cpu().numpy() - want) ** 2).mean() / (want ** 2).mean())


@pytest.mark.parametrize("M,K,N", [(2048, 2048, 1), (2048, 5632, 3), (5632, 2048, 13), (1000, 4096, 40), (700, 2048, 500)])
def test_mean_error_of_the_products(gq_lib, cuda_dev, M, K, N):
    blocks = weights(M, K, 4)
    x = np.random.default_rng(N).standard_normal((N, K), np.float32)
    q, xs = torch.from_numpy(blocks).to(cuda_dev), torch.from_numpy(x).to(cuda_dev)
    w = ref.weights("mxfp4", blocks, M, K)[0]
    assert off(gq_lib.mul_mat(q, "mxfp4", M, K, xs), x.astype(np.float64) @ w.T) <= LIMIT
    assert off(gq_lib.mul_mat_mx4x(q, "mxfp4", M, K, xs), ref.mx_values(*ref.mx_quantize(x)) @ w.T) <= LIMIT


@pytest.mark.parametrize("t", ("q4_0", "q8_0", "q4_k", "mxfp4"))
@pytest.mark.parametrize("E,N,k", [(4, 1, 2), (8, 16, 2), (2, 40, 2)])
def test_mean_error_of_the_expert_layer(gq_lib, cuda_dev, t, E, N, k):
    layer = Layer(gq_lib, cuda_dev, t, E, 2048, 1024)
    x, ids, w = layer.inputs(N, k)
    x = np.random.default_rng(N).standard_normal(x.shape).astype(np.float32)
    want, _ = ref.moe(*layer.ref, x.astype(np.float64), ids, w)
    assert off(layer.run(x, ids, w), want) <= LIMIT


@pytest.mark.parametrize("M,K", [(2048, 2048), (5632, 544), (300, 4096)])
@pytest.mark.parametrize("N", [12, 15, 16, 17, 18, 24])
def test_both_sides_of_the_token_border(gq_lib, cuda_dev, M, K, N):
    """Up to 16 tokens the workspace holds split activations alone, from 17 the weights' records, too."""
    laid_out = gq_lib.mx4x_workspace_size("mxfp4", M, K, N) >= M * K // 2
    assert laid_out == (N >= 17)
    blocks = weights(M, K, 5)
    x = np.random.default_rng(N).standard_normal((N, K), np.float32)
    y = gq_lib.mul_mat_mx4x(torch.from_numpy(blocks).to(cuda_dev), "mxfp4", M, K, torch.from_numpy(x).to(cuda_dev))
    want, tol = ref.product(*ref.weights("mxfp4", blocks, M, K), ref.mx_values(*ref.mx_quantize(x)))
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
