"""A call that CUDA refuses reports it once: nothing is left behind for the next launch, the
library's or the program's, to find."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

A256 = 0x7000_0000_0000   # not memory: the calls end before anything reads it


def launches_still_work(gq_lib, dev):
    assert (torch.ones(8, device=dev) * 2).sum().item() == 16
    q = gq_lib.quantize(torch.ones((4, 32), device=dev), "mxfp4")
    assert (gq_lib.dequantize(q, "mxfp4", 4, 32) == 1).all()


def test_no_memory_for_the_workspace(gq_lib, cuda_dev):
    """2 TB and more: no device has them."""
    lib, n = gq_lib.lib, 1 << 20
    assert lib.gq_mul_mat(A256, gq_lib.Q4_0, 256, n, A256, n, A256, None) == -5
    launches_still_work(gq_lib, cuda_dev)
    assert lib.gq_mul_mat_mx4x(A256, gq_lib.MXFP4, 1 << 17, 1 << 23, A256, 1 << 17, A256, None) == -5
    launches_still_work(gq_lib, cuda_dev)


def test_legacy_stream_during_a_capture(gq_lib, cuda_dev):
    """While a blocking stream is captured, the legacy stream cannot be used. The capture goes on."""
    box = ctypes.c_uint64()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(box))) == 0
    blocking = torch.cuda.ExternalStream(box.value)
    q = gq_lib.quantize(torch.ones((64, 64), device=cuda_dev), "mxfp4")
    x, y = torch.ones((2, 64), device=cuda_dev), torch.zeros((2, 64), device=cuda_dev)
    ws = torch.empty(gq_lib.workspace_size("mxfp4", 64, 64, 2), dtype=torch.uint8, device=cuda_dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=blocking):
        gq_lib.mul_mat_ws(q, "mxfp4", 64, 64, x, ws, out=y)
        for f in (gq_lib.mul_mat, gq_lib.mul_mat_mx4x):
            with pytest.raises(gq_lib.GQError):
                f(q, "mxfp4", 64, 64, x, out=y, stream=torch.cuda.default_stream())
            y += 1
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 66).all()
    launches_still_work(gq_lib, cuda_dev)
