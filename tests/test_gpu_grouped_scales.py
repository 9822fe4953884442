"""Grouped products of weights whose blocks have scales far apart, where the block of the largest scale adds
nothing to the result: its codes are zeros, or its x. Every form of the kernels (few, some and many rows)."""
import numpy as np
import pytest
import torch

import grouped_reference as gr
import mx_reference as ref
from test_gpu_grouped import near

pytestmark = pytest.mark.gpu

# What the two terms of a weight may lose, in parts of the largest scale of its 128 (256) weights. The scale is
# brought to fp16 under a power of two that puts the largest at 2^14 (Q4_K: 2^12 at least) and the codes into
# [-1, 1], so a scale among fp16's subnormals is off by 2^-25, and so are the two terms: 2^-24 of a weight whose
# unit is 2^7 (Q8_0), 2^11 (Q4_0) or at least 2^8 (Q4_K) of the largest scale; that is 2^-31, 2^-35, 2^-32. MXFP4:
# a block 2^-37 below the largest is lost, up to 6 2^-37. Half of each is left for what the sums lose of subnormal
# terms: 26 instructions of 19 units of 2^-24 of 2^-14 |x|, 2^-36 of the largest scale at most.
LOST = {"q4_0": 2.0 ** -34, "q8_0": 2.0 ** -30, "q4_k": 2.0 ** -31, "mxfp4": 2.0 ** -34}
M = 96


def bound(t, w, z, d, x):
    ax, a = np.abs(x), np.abs(w) + z
    most = np.maximum(ax.max(1, keepdims=True), 2.0 ** -110)
    return (w.shape[1] / 32 + 520) * ref.EPS * (ax @ a.T) + 2.0 ** -38 * most * a.sum(1) + LOST[t] * (ax @ d.T)


def halves(d):
    return np.ascontiguousarray(d.astype(np.float16))[..., None].view(np.uint8)


def small(rng, shape):
    """fp16 scales from the smallest subnormal to 2^-4, all bits in use."""
    d = np.ldexp(1 + rng.integers(0, 1024, shape) / 1024, rng.integers(-24, -4, shape))
    return d.astype(np.float16)


def blocks(t, K, rng):
    """(bytes, where a weight's block is the large one)."""
    n = K // 32
    at = rng.integers(0, 4, (M, (n + 3) // 4))                      # of each 128 weights
    large = (np.arange(n) % 4 == np.repeat(at, 4, axis=1)[:, :n])
    if t == "mxfp4":
        codes = rng.integers(0, 16, (M, n, 32)).astype(np.uint8)
        scales = 190 - rng.integers(20, 45, (M, n))                 # 2^-20 to 2^-44 of the large one
        codes[large] = 0
        return ref.mx_pack(codes, np.where(large, 190, scales).astype(np.uint8)), large
    d = small(rng, (M, n))
    d[large] = np.ldexp(1 + rng.integers(0, 1024, (M, n)) / 1024, rng.integers(4, 16, (M, n)))[large]
    if t == "q8_0":
        c = rng.choice(np.array([-127, -126, -65, 3, 101, 127]), (M, n, 32))
        c[large] = 0
        q = c.astype(np.int8).view(np.uint8)
    else:
        c = rng.choice(np.array([0, 1, 3, 7, 9, 15]), (M, n, 32))
        c[large] = 8
        q = (c[..., :16] | (c[..., 16:] << 4)).astype(np.uint8)
    return np.concatenate([halves(d), q], -1).reshape(M, -1), large


def superblocks(K, rng):
    """Q4_K: one sub-block of each eight has the largest scale and min (and codes 0), the others small scales; in
    every second super-block the smallness comes from d against dmin, mins only in the large one."""
    n = K // 256
    large = np.arange(8) == rng.integers(0, 8, (M, n, 1))
    far = (np.arange(n) % 2 == 0)[None, :, None]
    sc = np.where(large, 63, np.where(far, rng.integers(1, 64, (M, n, 8)), rng.integers(0, 3, (M, n, 8))))
    m = np.where(large, 63, np.where(far, 0, rng.integers(0, 64, (M, n, 8))))
    d = np.where(far[..., 0], small(rng, (M, n)), np.ldexp(1 + rng.integers(0, 1024, (M, n)) / 1024, 15))
    dmin = np.ldexp(1 + rng.integers(0, 1024, (M, n)) / 1024, np.where(far[..., 0], 15, -20))
    s = np.zeros((M, n, 12), np.uint8)
    s[..., :4] = sc[..., :4] | (sc[..., 4:] >> 4 << 6)
    s[..., 4:8] = m[..., :4] | (m[..., 4:] >> 4 << 6)
    s[..., 8:] = (sc[..., 4:] & 15) | ((m[..., 4:] & 15) << 4)
    q = rng.integers(0, 16, (M, n, 8, 32))
    q[np.broadcast_to(large[..., None], q.shape)] = 0
    q = q.reshape(M, n, 4, 2, 32)
    q = (q[..., 0, :] | (q[..., 1, :] << 4)).astype(np.uint8).reshape(M, n, 128)
    return np.concatenate([halves(d), halves(dmin), s, q], -1).reshape(M, -1), large.reshape(M, -1)


@pytest.mark.parametrize("n", [9, 40, 130])
@pytest.mark.parametrize("t,K", [("q4_0", 512), ("q4_0", 480), ("q8_0", 512), ("q8_0", 480), ("q4_k", 512),
                                 ("mxfp4", 512), ("mxfp4", 480)])
def test_small_scales_beside_a_large_one(gq_lib, cuda_dev, t, K, n):
    rng = np.random.default_rng(K + n)
    raw, large = superblocks(K, rng) if t == "q4_k" else blocks(t, K, rng)
    w = gr.weights(t, raw, M, K)
    blk = np.zeros((n, K // 32, 32))
    # a token stands for a weight row: x is zero in the row's large blocks, in every third also but in one block
    for i in range(n):
        live = ~large[i % M]
        if i % 3 == 2:
            live = live & (np.arange(K // 32) == rng.choice(np.flatnonzero(live)))
        blk[i] = live[:, None] * (rng.standard_normal(32) if i % 3 == 0 else 1.0)
    x = blk.reshape(n, K).astype(np.float32)
    off = torch.tensor([0, n], dtype=torch.int32, device=cuda_dev)
    y = gq_lib.mul_mat_grouped(torch.from_numpy(np.ascontiguousarray(raw)).to(cuda_dev), t, 1, M, K,
                               torch.from_numpy(x).to(cuda_dev), off)
    x = x.astype(np.float64)
    near(y, x @ w[0].T, bound(t, *w, x))


def by_hand(t):
    """(bytes of a row, K): a largest scale for the first block (Q4_K: two), and scales whose rounding goes the same
    way in all other weights."""
    one = lambda v: halves(np.array([v]))[0]
    if t == "q8_0":      # 1.5 2^-16 under 2^-8, a tie between multiples of 2^-24
        d, codes = [32768.0] + [1.5 * 2.0 ** -16] * 3, [0] + [127] * 3
        return np.concatenate([np.concatenate([one(v), np.full(32, c, np.uint8)]) for v, c in zip(d, codes)]), 128
    if t == "q4_0":      # 1.5 2^-20 under 2^-4
        d, codes = [32768.0] + [1.5 * 2.0 ** -20] * 3, [0x88] + [0] * 3
        return np.concatenate([np.concatenate([one(v), np.full(16, c, np.uint8)]) for v, c in zip(d, codes)]), 128
    if t == "mxfp4":     # 2^-37 of the largest
        return np.concatenate([np.concatenate([[s], np.full(16, c)]) for s, c in
                               ((190, 0x00), (153, 0x77), (153, 0x77), (153, 0x77))]).astype(np.uint8), 128
    # mins 32 and 31 (an OR of 63) of 2^15: 2^-14 goes under 2^-11
    s = np.array([0, 0, 1, 1, 32, 31, 0, 0, 1, 1, 1, 1], np.uint8)
    return np.concatenate([one(2.0 ** -14), one(32768.0), s, np.full(32, 0, np.uint8), np.full(96, 0xFF, np.uint8)]), 256


@pytest.mark.parametrize("n", [9, 40, 130])
@pytest.mark.parametrize("t", ["q4_0", "q8_0", "q4_k", "mxfp4"])
def test_by_hand(gq_lib, cuda_dev, t, n):
    row, K = by_hand(t)
    raw = np.tile(row, (M, 1))
    w = gr.weights(t, raw, M, K)
    x = np.ones((n, K), np.float32)
    x[:, :64 if t == "q4_k" else 32] = 0
    off = torch.tensor([0, n], dtype=torch.int32, device=cuda_dev)
    y = gq_lib.mul_mat_grouped(torch.from_numpy(raw).to(cuda_dev), t, 1, M, K, torch.from_numpy(x).to(cuda_dev), off)
    x = x.astype(np.float64)
    near(y, x @ w[0].T, bound(t, *w, x))
