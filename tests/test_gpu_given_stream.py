"""Calls with `stream=` and no `out`: the result is in memory that nothing queued elsewhere uses."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DELAY = 200_000_000   # clock cycles, about 0.1 s: longer than everything the host does meanwhile


def entries(gq_lib, dev):
    """name -> f(scale, **kw), whose result depends on scale."""
    M = K = 512
    N = 2048
    g = torch.Generator(device=dev).manual_seed(0)
    W = torch.randn((M, K), device=dev, generator=g)
    q = {t: gq_lib.quantize(W, t) for t in ("mxfp4", "q4_0")}
    x = {s: torch.randn((N, K), device=dev, generator=g) * s for s in (1.0, 2.0)}
    z = {s: torch.randn((N, 128), device=dev, generator=g) * s for s in (1.0, 2.0)}
    w = {s: torch.randn((4096, K), device=dev, generator=g) * s for s in (1.0, 2.0)}
    few = {s: v[:2].contiguous() for s, v in x.items()}
    m = {s: v[:64].contiguous() for s, v in x.items()}
    gamma = torch.ones(K, device=dev)
    parts = [gq_lib.quantize(torch.randn((4 * 512, 512), device=dev, generator=g), "q4_0") for _ in range(3)]
    layer = gq_lib.MoeExperts(*parts, "q4_0", 4, 512, 512)
    ids = torch.randint(0, 4, (64, 2), device=dev, generator=g, dtype=torch.int32)
    wts = torch.rand((64, 2), device=dev, generator=g)
    blocks = {s: gq_lib.quantize(w[s], "mxfp4") for s in w}
    torch.cuda.synchronize()
    return {
        "quantize": lambda s, **kw: gq_lib.quantize(w[s], "mxfp4", **kw),
        "dequantize": lambda s, **kw: gq_lib.dequantize(blocks[s], "mxfp4", 4096, K, **kw),
        "mul_mat": lambda s, **kw: gq_lib.mul_mat(q["mxfp4"], "mxfp4", M, K, x[s], **kw),
        "mul_mat q4_0": lambda s, **kw: gq_lib.mul_mat(q["q4_0"], "q4_0", M, K, x[s], **kw),
        "noalloc": lambda s, **kw: gq_lib.mul_mat_noalloc(q["mxfp4"], "mxfp4", M, K, x[s], **kw),
        "q8x": lambda s, **kw: gq_lib.mul_mat_q8x(q["q4_0"], "q4_0", M, K, few[s], **kw),
        "rmsnorm": lambda s, **kw: gq_lib.mul_mat_rmsnorm(q["mxfp4"], "mxfp4", M, K, x[s], gamma, 1e3, **kw),
        "swiglu": lambda s, **kw: gq_lib.mul_mat_swiglu(q["mxfp4"], q["mxfp4"], "mxfp4", M, K, x[s], **kw),
        "mx4x": lambda s, **kw: gq_lib.mul_mat_mx4x(q["mxfp4"], "mxfp4", M, K, x[s], **kw),
        "moe_route": lambda s, **kw: gq_lib.moe_route(z[s], 8, **kw)[1],
        "moe_swiglu": lambda s, **kw: gq_lib.moe_swiglu(layer, m[s], ids, wts, **kw),
    }


NAMES = ("quantize", "dequantize", "mul_mat", "mul_mat q4_0", "noalloc", "q8x", "rmsnorm", "swiglu", "mx4x",
         "moe_route", "moe_swiglu")


@pytest.fixture(scope="module")
def run(gq_lib, cuda_dev):
    return entries(gq_lib, cuda_dev)


@pytest.mark.parametrize("name", NAMES)
def test_freed_memory_in_use_on_the_current_stream(run, cuda_dev, name):
    f = run[name]
    want = f(1.0)
    torch.cuda.synchronize()
    old = torch.full_like(want, 5)
    copy = torch.empty_like(want)
    side = torch.cuda.Stream()
    f(1.0, stream=side)            # the library has its workspace for `side`
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    copy.copy_(old)
    del old                        # its block is the current stream's next one of this size
    got = f(1.0, stream=side)
    torch.cuda.synchronize()
    assert (copy == 5).all() and torch.equal(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_result_in_use_on_the_current_stream(run, cuda_dev, name):
    f = run[name]
    want = f(1.0), f(2.0)
    copy = torch.empty_like(want[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = f(1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(DELAY)
    copy.copy_(got)
    del got                        # the current stream reads it later than `side` could write it again
    again = f(2.0, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want[0]) and torch.equal(again, want[1])


def test_uploaded_tensor(gq_lib, cuda_dev, tmp_path):
    import gguf_writer
    from block_quantized_matmul_gq_gb300 import gguf
    data = bytes(range(256)) * (1 << 14)
    raw, _ = gguf_writer.build([], [("w", (len(data) // 4,), 0, data)])
    (tmp_path / "w.gguf").write_bytes(raw)
    side = torch.cuda.Stream()
    with gguf.GGUFFile(str(tmp_path / "w.gguf")) as file:
        old = torch.full((len(data),), 5, dtype=torch.uint8, device=cuda_dev)
        copy = torch.empty_like(old)
        torch.cuda.synchronize()
        torch.cuda._sleep(DELAY)
        copy.copy_(old)
        del old
        got = file.upload("w", cuda_dev, stream=side)
        torch.cuda.synchronize()
    assert (copy == 5).all() and bytes(got.cpu().numpy()) == data
