"""The workspaces that the library owns: one call's at a time, of one stream, whatever that
stream's handle says, and there as long as a graph has its address."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

PER_THREAD = 2   # cudaStreamPerThread: one handle, another stream in every thread


class Handle:
    """A stream by its bare handle, as a C caller passes it."""

    def __init__(self, handle):
        self.cuda_stream = handle


def calls(gq_lib, dev, seed):
    """Calls f(stream, out) that use the library's workspaces, on inputs of this seed, and each
    one's result by itself."""
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, device=dev, generator=g)
    M, K, D, F, E = 512, 1024, 256, 512, 6
    w = {t: gq_lib.quantize(rand(M, K) * 0.05, t) for t in ("mxfp4", "q4_0", "q4_k")}
    x = {n: rand(n, K) for n in (3 + seed, 8 + seed, 90 + 8 * seed)}
    few, some, many = x.values()
    layer = gq_lib.MoeExperts(gq_lib.quantize(rand(E * F, D) * 0.05, "q4_0"),
                              gq_lib.quantize(rand(E * F, D) * 0.05, "q4_0"),
                              gq_lib.quantize(rand(E * D, F) * 0.05, "q4_0"), "q4_0", E, D, F)
    xm, wm = rand(9 + seed, D), torch.rand((9 + seed, 2), device=dev, generator=g)
    ids = torch.randint(0, E, (9 + seed, 2), device=dev, generator=g, dtype=torch.int32)
    todo = [lambda s, o, x=x, t=t: gq_lib.mul_mat(w[t], t, M, K, x, out=o, stream=s)
            for t, x in (("mxfp4", few), ("mxfp4", many), ("q4_0", some), ("q4_0", many), ("q4_k", many))]
    todo += [lambda s, o, x=x: gq_lib.mul_mat_mx4x(w["mxfp4"], "mxfp4", M, K, x, out=o, stream=s) for x in (few, many)]
    todo += [lambda s, o: gq_lib.moe_swiglu(layer, xm, ids, wm, out=o, stream=s),
             lambda s, o: gq_lib.mul_mat_swiglu(w["q4_0"], w["q4_0"], "q4_0", M, K, many, out=o, stream=s)]
    want = [f(None, None) for f in todo]
    torch.cuda.synchronize()
    return todo, want


def run_threads(work, stream_of, rounds):
    """Every thread its own calls, all at once; whether each result is the one by itself."""
    outs = [[[torch.zeros_like(w) for w in want] for _ in range(rounds)] for _, want in work]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(work)), []

    def run(i):
        try:
            stream = stream_of(i)
            start.wait()
            for out in outs[i]:
                for f, o in zip(work[i][0], out):
                    f(stream, o)
        except Exception as e:   # shown by the assertion below
            failed.append(e)
            start.abort()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for (_, want), rounds_of in zip(work, outs):
        for out in rounds_of:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_threads_on_the_per_thread_stream(gq_lib, cuda_dev):
    run_threads([calls(gq_lib, cuda_dev, i) for i in range(4)], lambda i: Handle(PER_THREAD), 12)
    assert gq_lib.get_last_error() == 0


def test_threads_on_one_stream(gq_lib, cuda_dev):
    shared = torch.cuda.Stream()
    run_threads([calls(gq_lib, cuda_dev, i) for i in range(4)], lambda i: Handle(shared.cuda_stream), 12)
    assert gq_lib.get_last_error() == 0


class OwnStream:
    """A stream that is destroyed at once, with its work still queued."""

    def __enter__(self):
        box = ctypes.c_uint64()
        assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(box))) == 0
        self.handle = box.value
        return Handle(self.handle)

    def __exit__(self, *exc):
        assert int(torch.cuda.cudart().cudaStreamDestroy(self.handle)) == 0


def test_streams_destroyed_with_work_queued(gq_lib, cuda_dev):
    """A destroyed stream's handle may be the next one's while its kernels still run."""
    work = [calls(gq_lib, cuda_dev, i) for i in range(2)]
    turns = [(work[n % 2], n // 2 % len(work[0][0])) for n in range(300)]
    outs = [(torch.zeros_like(want[k]), want[k]) for (_, want), k in turns]
    torch.cuda.synchronize()
    for ((todo, _), k), (out, _) in zip(turns, outs):
        with OwnStream() as stream:
            todo[k](stream, out)
            todo[k](stream, out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs) and gq_lib.get_last_error() == 0


def test_a_captured_workspace_stays(gq_lib, cuda_dev):
    """The tensor-core paths may be captured with the library's workspace once it is large enough:
    later, larger calls and other streams leave the graph's address alone."""
    M, K, N = 256, 512, 96
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    q = gq_lib.quantize(torch.randn((M, K), device=cuda_dev, generator=g), "q4_0")
    x = torch.randn((N, K), device=cuda_dev, generator=g)
    big = torch.randn((20 * N, K), device=cuda_dev, generator=g)
    want, want_big = gq_lib.mul_mat(q, "q4_0", M, K, x), gq_lib.mul_mat(q, "q4_0", M, K, big)
    out, side = torch.zeros((N, M), device=cuda_dev), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        gq_lib.mul_mat(q, "q4_0", M, K, x, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gq_lib.mul_mat(q, "q4_0", M, K, x, out=out)
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got_big = gq_lib.mul_mat(q, "q4_0", M, K, big)
        scratch = torch.full((N * K * 2,), 255, dtype=torch.uint8, device=cuda_dev)
        graph.replay()
    for _ in range(30):
        with OwnStream() as stream:
            gq_lib.mul_mat(q, "q4_0", M, K, x, out=torch.empty_like(out), stream=stream)
            torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(got_big, want_big) and (scratch == 255).all()


def test_calls_while_another_thread_captures(gq_lib, cuda_dev):
    """Eager calls of one thread leave the capture of another alone, and the other way round."""
    todo, want = calls(gq_lib, cuda_dev, 0)
    eager, captured = [[torch.zeros_like(w) for w in want] for _ in range(2)]
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    ws = torch.empty(gq_lib.workspace_size("mxfp4", 64, 64, 2), dtype=torch.uint8, device=cuda_dev)
    q, x = gq_lib.quantize(torch.ones((64, 64), device=cuda_dev), "mxfp4"), torch.ones((2, 64), device=cuda_dev)
    y, wrong = torch.zeros((2, 64), device=cuda_dev), []
    tensor_cores = [2, 3, 4, 8]   # the calls that may be captured with the library's workspace
    for s in (stream, side):
        for f, o in zip(todo, eager):
            f(s, o)
    torch.cuda.synchronize()
    for o in eager:
        o.zero_()
    torch.cuda.synchronize()

    def run():
        try:
            for f, o in zip(todo, eager):
                f(stream, o)
        except Exception as e:
            wrong.append(e)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gq_lib.mul_mat_ws(q, "mxfp4", 64, 64, x, ws, out=y)
        thread = threading.Thread(target=run)
        thread.start()
        thread.join()
        for i in tensor_cores:
            todo[i](None, captured[i])
    graph.replay()
    torch.cuda.synchronize()
    assert not wrong and (y == 64).all()
    assert all(torch.equal(a, b) for a, b in zip(eager, want))
    assert all(torch.equal(captured[i], want[i]) for i in tensor_cores)
