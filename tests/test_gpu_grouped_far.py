"""Grouped products at sizes that pass 32 bits, or 40."""
import pytest
import torch

import grouped_reference as gr
from test_gpu_grouped import near

pytestmark = pytest.mark.gpu


def test_many_tokens_and_weight_rows(gq_lib, cuda_dev):
    """N * E * M above 2^40: only R * M has to be in range."""
    experts, M, K, R = 1024, 4096, 32, (1 << 18) + 1000
    W = gq_lib.quantize(torch.randn((experts * M, K), device=cuda_dev) * 0.05, "q8_0")
    assert R * experts * M > 2 ** 40
    x = torch.randn((R, K), device=cuda_dev)
    off = (torch.arange(experts + 1, device=cuda_dev) * R // experts).int()
    y = gq_lib.mul_mat_grouped(W, "q8_0", experts, M, K, x, off)
    for e in (0, 500, experts - 1):
        a, b = int(off[e]), int(off[e]) + 5
        w = gr.weights("q8_0", W[e * M:(e + 1) * M].cpu().numpy(), M, K)
        near(y[a:b], *gr.product(*w, x[a:b].cpu().double().numpy()))
