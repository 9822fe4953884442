"""Plain 64-bit implementations that the MXFP4 and mixture-of-experts tests compare with
(numpy; nothing of the library), and the error bounds that include/gq.h states."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EPS = 2.0 ** -24


def mx_quantize(W):
    """(codes 0..15, scale bytes) of 32-value blocks of W (..., K fp32)."""
    v = np.asarray(W, np.float32).reshape(*W.shape[:-1], -1, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.abs(np.where(bad[..., None], 0.0, v).astype(np.float64))
    amax = a.max(-1)
    e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127)
    e = np.clip(e, -127, 127)
    a = np.ldexp(a, -e[..., None])
    dist = np.abs(a[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    near = dist == best                       # two of them at a tie: the even code
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    code = code + 8 * np.signbit(v)
    return np.where(bad[..., None], 0, code).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx_pack(codes, scales):
    q = (codes[..., :16] | (codes[..., 16:] << 4)).astype(np.uint8)
    b = np.concatenate([scales[..., None], q], -1)
    return np.ascontiguousarray(b.reshape(*b.shape[:-2], -1))


def mx_values(codes, scales):
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    v = v * s[..., None]
    return v.reshape(*v.shape[:-2], -1)


def mx_unpack(blocks):
    b = blocks.reshape(*blocks.shape[:-1], -1, 17)
    q = b[..., 1:]
    return np.concatenate([q & 15, q >> 4], -1), b[..., 0]


def weights(t, blocks, M, K):
    """(What, |dmin m| per weight: what Q4_K takes off every code) in 64 bits."""
    import oracle
    if t == "mxfp4":
        w = mx_values(*mx_unpack(blocks.reshape(M, -1)))
        return w, np.zeros_like(w)
    w = oracle.dequantize(t, blocks, M, K).astype(np.float64)
    if t == "q4_k":   # the min is What of code 0
        b = blocks.reshape(M, -1, 144).copy()
        b[:, :, 16:] = 0
        return w, np.abs(oracle.dequantize(t, b.reshape(M, -1), M, K).astype(np.float64))
    return w, np.zeros_like(w)


def product(w, z, x):
    """(Y, bound) of Y = x . w^T: roundings of the fp32 sums, and of the two terms of x, which
    keep 22 bits of an element down to 2^-39 of the largest."""
    c = (w.shape[1] / 32 + 160) * EPS
    a = np.abs(w) + z
    return x @ w.T, c * (np.abs(x) @ a.T) + 2.0 ** -38 * np.abs(x).max(1, keepdims=True) * a.sum(1)


def route(logits, top_k, renorm):
    z = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    ids = np.argsort(-z, axis=1, kind="stable")[:, :top_k]
    top = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(z == top, 1.0, np.exp(z - top))
    sel = np.take_along_axis(p, ids, 1)
    w = sel / (sel if renorm else p).sum(1, keepdims=True)
    return ids.astype(np.int32), np.where(top == -np.inf, 0.0, w)


def moe(gate, up, down, x, ids, wts):
    """(Y, bound); gate, up, down: lists over experts of (What, z)."""
    N, D = x.shape
    y, tol = np.zeros((N, D)), np.zeros((N, D))
    for n in range(N):
        for j in range(ids.shape[1]):
            e = ids[n, j]
            if not 0 <= e < len(gate):
                continue
            g, eg = product(*gate[e], x[n:n + 1])
            u, eu = product(*up[e], x[n:n + 1])
            s = g / (1 + np.exp(-g))
            h = s * u
            # |Swish'| <= 1.1, the products of the two errors, expf, division and product
            eh = 1.1 * (np.abs(u) + eu) * eg + np.abs(s) * eu + 16 * EPS * np.abs(h)
            o, eo = product(*down[e], h)
            eo = eo * 1.01 + eh @ np.abs(down[e][0]).T
            w = float(wts[n, j])
            y[n] += w * o[0]
            tol[n] += abs(w) * (eo[0] + ids.shape[1] * 2 * EPS * np.abs(o[0]))
    return y, tol
