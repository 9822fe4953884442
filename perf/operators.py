"""What is measured of the microscaled 4-bit (MXFP4) product and the mixture-of-experts layer.

Five calls, each in a plain form (elementary torch operations in 32 bits, in 64 where values
lie next to a rounding border) and, where `own` is true, as a user calls libgq:

  quantize   W (M x K fp32) -> MXFP4 blocks and back: per 32 weights e = floor(log2 amax) - 2,
             scale 2^e, codes E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and the negatives), nearest even
  product    Y = X . What^T with MXFP4 weights and fp32 X
  mx_product Y = Xhat . What^T, X quantized to MXFP4 the same way within the call
  route      router logits (N x E) -> the top_k experts of each token, and their weights
  moe        Y[n] = sum_j w[n,j] Wdown_e (Swish(Wgate_e x_n) * (Wup_e x_n)), e = ids[n,j]

A case is a dict of plain values; inputs come from the seed alone.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"q4_0": (32, 18), "q8_0": (32, 34), "q4_k": (256, 144), "mxfp4": (32, 17)}


def listed():
    return [
        # a small projection quantized on its own when a model is loaded: the launch counts
        dict(name="quantize kv projection", op="quantize", M=256, K=2048),
        # the vocabulary matrix at load time: the largest matrix of a small model
        dict(name="quantize vocabulary", op="quantize", M=32000, K=2048),
        # one token through an attention projection: the smallest call of a decode step
        dict(name="product 1 token", op="product", M=2048, K=2048, N=1),
        # a ragged batch of decoding sequences through the vocabulary matrix
        dict(name="product 13 tokens", op="product", M=32000, K=2048, N=13),
        # prompt tokens through a feed-forward matrix
        dict(name="mx product prompt", op="mx_product", M=5632, K=2048, N=512),
        # a long prompt through a larger model's feed-forward matrix: the largest product
        dict(name="mx product long prompt", op="mx_product", M=11008, K=4096, N=2048),
        # one decoding token's router
        dict(name="route 1 token", op="route", N=1, E=64, top_k=4, renorm=True, masked=False),
        # the routers of a whole prompt, some experts masked away
        dict(name="route prompt", op="route", N=8191, E=128, top_k=8, renorm=True, masked=True),
        # one token, few experts with the feed-forward width split between them
        dict(name="moe 1 token q4_0", op="moe", t="q4_0", N=1, E=8, top_k=2, D=2048, F=1408),
        # a small batch over microscaled experts
        dict(name="moe 4 tokens mxfp4", op="moe", t="mxfp4", N=4, E=32, top_k=4, D=2048, F=1408),
        # a batch of decoding sequences, 8-bit experts of an odd number of blocks
        dict(name="moe 16 tokens q8_0", op="moe", t="q8_0", N=16, E=64, top_k=8, D=2048, F=704),
        # a larger batch, every expert at work
        dict(name="moe 61 tokens q4_k", op="moe", t="q4_k", N=61, E=64, top_k=8, D=2048, F=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "mx_product", "mx_product", "route", "moe", "moe", "moe"))
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 16000), K=32 * _log(rng, 1, 128))
    if op == "product":
        return dict(op=op, M=_log(rng, 1, 32000), K=32 * _log(rng, 1, 176), N=_log(rng, 1, 64))
    if op == "mx_product":
        return dict(op=op, M=_log(rng, 1, 11008), K=32 * _log(rng, 1, 128), N=_log(rng, 1, 2048))
    if op == "route":
        E = _log(rng, 2, 512)
        return dict(op=op, N=_log(rng, 1, 8192), E=E, top_k=rng.randint(1, min(E, 16)), renorm=rng.random() < 0.7,
                    masked=rng.random() < 0.5)
    t = rng.choice(("q4_0", "q8_0", "q4_k", "mxfp4"))
    unit = 256 if t == "q4_k" else 32
    E = _log(rng, 2, 64)
    return dict(op=op, t=t, N=_log(rng, 1, 61), E=E, top_k=rng.randint(1, min(E, 8)),
                D=unit * _log(rng, 1, 2048 // unit), F=unit * _log(rng, 1, 1024 // unit))


# ---- inputs -------------------------------------------------------------------------------


def _device():
    return torch.device("cuda:0")


def _mx_parts(W):
    """E2M1 codes (0..15) and shared exponents of 32-value blocks of W; zero blocks: exponent -127."""
    v = W.reshape(*W.shape[:-1], -1, 32).double()
    amax = v.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = torch.ldexp(v.abs(), -e.double().unsqueeze(-1))
    code = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() \
        + (a >= 3.5).int() + (a > 5.0).int()
    return code + 8 * torch.signbit(v).int(), e


def _mx_values(code, e):
    grid = torch.tensor(GRID, dtype=torch.float64, device=code.device)
    v = grid[(code & 7).long()] * (1 - 2 * (code >> 3)).double()
    return torch.ldexp(v, e.double().unsqueeze(-1)).float().flatten(-2)


def _halves(code):
    """32 4-bit codes -> 16 bytes: element j in the low nibble of byte j, j + 16 in the high one."""
    return (code[..., :16] | (code[..., 16:] << 4)).to(torch.uint8)


def _blocks(t, shape, g):
    """Block bytes of weights like N(0, 0.02): (..., row bytes) for a shape (..., K)."""
    dev = _device()
    K = shape[-1]
    if t == "mxfp4":
        code, e = _mx_parts(torch.randn(shape, generator=g, device=dev) * 0.02)
        return torch.cat([(e + 127).to(torch.uint8).unsqueeze(-1), _halves(code)], -1).flatten(-2)
    if t == "q4_k":
        head = (*shape[:-1], K // 256)
        d = (torch.rand(head, generator=g, device=dev) * 1e-4 + 1e-4).half()
        dmin = (torch.rand(head, generator=g, device=dev) * 5e-4 + 1e-3).half()
        s = torch.randint(0, 256, (*head, 12), generator=g, device=dev).to(torch.uint8)
        q = (torch.randn((*head, 256), generator=g, device=dev) * 3.2 + 7.5).round().clamp(0, 15).int()
        q = q.view(*head, 4, 2, 32)
        q = (q[..., 0, :] | (q[..., 1, :] << 4)).to(torch.uint8).flatten(-2)
        return torch.cat([d.unsqueeze(-1).view(torch.uint8), dmin.unsqueeze(-1).view(torch.uint8), s, q], -1).flatten(-2)
    head = (*shape[:-1], K // 32)
    top = 0.02 * (1.7 + torch.rand(head, generator=g, device=dev))
    n = torch.randn((*head, 32), generator=g, device=dev)
    if t == "q4_0":
        d = (top / 7).half()
        q = _halves((n * 3.2).round().clamp(-8, 7).int() + 8)
    else:
        d = (top / 127).half()
        q = (n * 58).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return torch.cat([d.unsqueeze(-1).view(torch.uint8), q], -1).flatten(-2)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        s["W"] = torch.randn((case["M"], case["K"]), generator=g, device=dev) * 0.02
    elif op in ("product", "mx_product"):
        s["blocks"] = _blocks("mxfp4", (case["M"], case["K"]), g).contiguous()
        s["X"] = torch.randn((case["N"], case["K"]), generator=g, device=dev)
    elif op == "route":
        z = torch.randn((case["N"], case["E"]), generator=g, device=dev) * 2
        if case["masked"]:
            # coarse logits (equal ones occur), and experts that a token may not use
            z = torch.where(torch.rand(z.shape, generator=g, device=dev) < 0.3, -math.inf, (z * 8).round() / 8)
            z[torch.rand(z.shape[0], generator=g, device=dev) < 0.02] = -math.inf
        s["logits"] = z
    else:
        E, D, F, t = case["E"], case["D"], case["F"], case["t"]
        s["gate"] = _blocks(t, (E, F, D), g).contiguous()
        s["up"] = _blocks(t, (E, F, D), g).contiguous()
        s["down"] = _blocks(t, (E, D, F), g).contiguous()
        s["X"] = torch.randn((case["N"], D), generator=g, device=dev)
        z = torch.randn((case["N"], E), generator=g, device=dev)
        p, ids = torch.sort(torch.softmax(z, -1), dim=-1, descending=True)
        p = p[:, : case["top_k"]]
        s["ids"] = ids[:, : case["top_k"]].int().contiguous()
        s["weights"] = (p / p.sum(-1, keepdim=True)).contiguous()
    return s


# ---- the passes ---------------------------------------------------------------------------


def _values(t, blocks):
    """fp32 weights (..., K) of block bytes (..., row bytes)."""
    n, nb = BLOCK[t]
    b = blocks.view(*blocks.shape[:-1], -1, nb)
    if t == "mxfp4":
        q = b[..., 1:].int()
        return _mx_values(torch.cat([q & 15, q >> 4], -1), b[..., 0].int() - 127)
    d = b[..., :2].contiguous().view(torch.float16).float()
    if t == "q8_0":
        return (b[..., 2:].contiguous().view(torch.int8).float() * d).flatten(-2)
    if t == "q4_0":
        q = b[..., 2:].int()
        return ((torch.cat([q & 15, q >> 4], -1) - 8).float() * d).flatten(-2)
    dmin = b[..., 2:4].contiguous().view(torch.float16).float()
    s = b[..., 4:16].int()
    lo, mid, hi = s[..., 0:4], s[..., 4:8], s[..., 8:12]
    sc = torch.cat([lo & 63, (hi & 15) | ((lo >> 6) << 4)], -1).float()
    mn = torch.cat([mid & 63, (hi >> 4) | ((mid >> 6) << 4)], -1).float()
    q = b[..., 16:].int().view(*b.shape[:-1], 4, 1, 32)
    q = torch.cat([q & 15, q >> 4], -2).flatten(-3, -2).float()
    return ((d * sc).unsqueeze(-1) * q - (dmin * mn).unsqueeze(-1)).flatten(-3)


def run(s):
    op = s["op"]
    if own:
        from block_quantized_matmul_gq_gb300 import binding

        if op == "quantize":
            b = binding.quantize(s["W"], "mxfp4")
            return binding.dequantize(b, "mxfp4", s["M"], s["K"])
        if op == "product":
            return binding.mul_mat(s["blocks"], "mxfp4", s["M"], s["K"], s["X"])
        if op == "mx_product":
            return binding.mul_mat_mx4x(s["blocks"], "mxfp4", s["M"], s["K"], s["X"])
        if op == "route":
            return binding.moe_route(s["logits"], s["top_k"], renorm=s["renorm"])
        experts = binding.MoeExperts(s["gate"], s["up"], s["down"], s["t"], s["E"], s["D"], s["F"])
        return binding.moe_swiglu(experts, s["X"], s["ids"], s["weights"])
    if op == "quantize":
        return _mx_values(*_mx_parts(s["W"]))
    if op == "product":
        return s["X"] @ _values("mxfp4", s["blocks"]).T
    if op == "mx_product":
        return _mx_values(*_mx_parts(s["X"])) @ _values("mxfp4", s["blocks"]).T
    if op == "route":
        z, ids = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
        top = z[:, :1]
        p = torch.where(top == -math.inf, 0.0, torch.exp(z - top))
        w = p[:, : s["top_k"]]
        total = (w if s["renorm"] else p).sum(-1, keepdim=True)
        return ids[:, : s["top_k"]].int(), torch.where(total > 0, w / total, 0.0)
    # every (token, expert) pair with its own copy of the expert's blocks
    ids = s["ids"].flatten().long()
    x = s["X"].repeat_interleave(s["top_k"], 0).unsqueeze(-1)
    g = torch.bmm(_values(s["t"], s["gate"][ids]), x)
    u = torch.bmm(_values(s["t"], s["up"][ids]), x)
    h = g / (1 + torch.exp(-g)) * u
    y = torch.bmm(_values(s["t"], s["down"][ids]), h).view(s["N"], s["top_k"], s["D"])
    return (y * s["weights"].unsqueeze(-1)).sum(1)


# ---- what a pass cannot do without --------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "route":
        n = case["N"] * case["E"]
        return dict(bytes=4 * n + 8 * case["N"] * case["top_k"], flops=2 * n)
    if op == "moe":
        E, D, F, N, k = case["E"], case["D"], case["F"], case["N"], case["top_k"]
        n, nb = BLOCK[case["t"]]
        active = E * (1 - (1 - k / E) ** N)  # experts that N tokens choose, each k of E
        return dict(bytes=active * 3 * D * F * nb / n + 8 * N * D + 8 * N * k, flops=6 * N * k * D * F)
    M, K = case["M"], case["K"]
    packed = M * K * 17 / 32
    if op == "quantize":  # to blocks, and from blocks to values
        return dict(bytes=8 * M * K + 2 * packed, flops=2 * M * K)
    N = case["N"]
    return dict(bytes=packed + 4 * N * K + 4 * N * M, flops=2 * M * K * N)


# ---- the definitions in 64 bits, apart from the forms above --------------------------------


def _nearest(W):
    """E2M1 times 2^e values of W (..., K) in 64 bits, by distance to the neighbouring grid values."""
    v = W.double().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -149)))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    scale = torch.exp2((e - 2).clamp(-127, 127))
    a = v.abs() / scale
    grid = torch.tensor(GRID, dtype=torch.float64, device=W.device)
    lo = (torch.searchsorted(grid, a.contiguous(), right=True) - 1).clamp(0, 7)
    hi = (lo + 1).clamp(max=7)
    down, up = a - grid[lo], grid[hi] - a
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)) | (lo == 7), lo, hi)
    return (torch.copysign(grid[pick], v) * scale).flatten(-2)


def _exact_weights(t, raw):
    """Weights in 64 bits from block bytes (rows, row bytes)."""
    n, nb = BLOCK[t]
    b = raw.reshape(raw.shape[0], -1, nb)

    def f16(at):
        w = b[:, :, at].long() | (b[:, :, at + 1].long() << 8)
        m, ex = (w & 1023).double(), (w >> 10) & 31
        mag = torch.where(ex == 0, m * 2.0 ** -24, (1024 + m) * torch.exp2(ex.double() - 25))
        return torch.where(w >= 32768, -mag, mag).unsqueeze(-1)

    if t == "q8_0":
        c = b[:, :, 2:].long()
        return (f16(0) * torch.where(c > 127, c - 256, c)).flatten(1)
    if t in ("q4_0", "mxfp4"):
        c = b[:, :, -16:].long()
        c = torch.cat([c % 16, c // 16], 2)
        if t == "q4_0":
            return (f16(0) * (c - 8)).flatten(1)
        table = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64, device=raw.device)
        return (table[c] * torch.exp2(b[:, :, :1].double() - 127)).flatten(1)
    out = torch.empty((raw.shape[0], b.shape[1], 256), dtype=torch.float64, device=raw.device)
    s = b[:, :, 4:16].long()
    for j in range(8):
        if j < 4:
            sc, mn = s[:, :, j] % 64, s[:, :, j + 4] % 64
        else:
            sc = s[:, :, j + 4] % 16 + 16 * (s[:, :, j - 4] // 64)
            mn = s[:, :, j + 4] // 16 + 16 * (s[:, :, j] // 64)
        c = b[:, :, 16 + 32 * (j // 2): 48 + 32 * (j // 2)].long()
        c = c // 16 if j % 2 else c % 16
        out[:, :, 32 * j: 32 * j + 32] = f16(0) * sc.unsqueeze(-1) * c - f16(2) * mn.unsqueeze(-1)
    return out.flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _nearest(s["W"])
    if op == "product":
        return s["X"].double() @ _exact_weights("mxfp4", s["blocks"]).T
    if op == "mx_product":
        return _nearest(s["X"]) @ _exact_weights("mxfp4", s["blocks"]).T
    if op == "route":
        z = s["logits"].double()
        # the place of expert e in its token's order: those above it, and equal ones before it
        E, k = case["E"], case["top_k"]
        ids = torch.empty((case["N"], k), dtype=torch.int32, device=z.device)
        left = z.clone()
        taken = torch.zeros_like(z, dtype=torch.bool)
        number = torch.arange(E, device=z.device).expand_as(z)
        for j in range(k):
            best = left.masked_fill(taken, -math.inf).amax(1, keepdim=True)
            first = torch.where((left == best) & ~taken, number, E).amin(1)
            ids[:, j] = first.int()
            taken.scatter_(1, first.unsqueeze(1), True)
        alive = (z > -math.inf).any(1, keepdim=True)
        share = torch.softmax(torch.where(alive, z, 0.0), 1) * alive
        w = share.gather(1, ids.long())
        if case["renorm"]:
            w = torch.where(alive, w / w.sum(1, keepdim=True), 0.0)
        return ids, w
    x, y = s["X"].double(), torch.zeros((case["N"], case["D"]), dtype=torch.float64, device=s["X"].device)
    for e in range(case["E"]):
        n, j = (s["ids"] == e).nonzero(as_tuple=True)
        if not n.numel():
            continue
        g = x[n] @ _exact_weights(case["t"], s["gate"][e]).T
        h = g * torch.sigmoid(g) * (x[n] @ _exact_weights(case["t"], s["up"][e]).T)
        o = h @ _exact_weights(case["t"], s["down"][e]).T
        y.index_add_(0, n, o * s["weights"][n, j].double().unsqueeze(-1))
    return y
