"""Grouped products whose weights begin behind 2^32 bytes, by every way that they are read, and of more tokens times
weight rows than 2^40."""
import numpy as np
import pytest
import torch

import grouped_reference as gr
from test_gpu_grouped import near, tokens

pytestmark = pytest.mark.gpu

E = 40
# rows of weights an expert; K by tensor maps and (4128) by copying warps
FAR = [("q4_0", 49152, 4096), ("q4_0", 49152, 4128), ("q8_0", 32768, 4128), ("q4_k", 49152, 4096),
       ("mxfp4", 53248, 4096), ("mxfp4", 53248, 4128)]


def last_expert(gq_lib, dev, t, M, K, nb, seed):
    W = torch.full((E * M, nb), 0x39, dtype=torch.uint8, device=dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    W[(E - 1) * M:] = gq_lib.quantize(torch.randn((M, K), device=dev, generator=g) * 0.05, t)
    assert (E - 1) * M * nb > 2 ** 32
    return W


@pytest.mark.parametrize("t,M,K", FAR)
def test_weights_behind_32_bits(gq_lib, cuda_dev, t, M, K):
    W = last_expert(gq_lib, cuda_dev, t, M, K, gq_lib.row_bytes(t, K), 1)
    some = torch.tensor([0, 1, 127, 128, 20000, M - 129, M - 1], device=cuda_dev)
    w = gr.weights(t, W[(E - 1) * M + some].cpu().numpy(), len(some), K)
    for R in (30, 1400, 5000):                      # few, some and many rows an expert
        x = torch.from_numpy(tokens(R, K)).to(cuda_dev)
        off = torch.zeros(E + 1, dtype=torch.int32, device=cuda_dev)
        off[E] = R
        y = gq_lib.mul_mat_grouped(W, t, E, M, K, x, off)
        near(y[R - 20:][:, some], *gr.product(*w, x[R - 20:].cpu().double().numpy()))
        del x, y


@pytest.mark.parametrize("t,M,K", [FAR[1], FAR[2], FAR[3], FAR[4]])
def test_swiglu_weights_behind_32_bits(gq_lib, cuda_dev, t, M, K):
    nb, R = gq_lib.row_bytes(t, K), 700
    gate, up = (last_expert(gq_lib, cuda_dev, t, M, K, nb, seed) for seed in (1, 2))
    some = torch.tensor([0, 63, 64, 20000, M - 65, M - 1], device=cuda_dev)
    wg, wu = (gr.weights(t, w[(E - 1) * M + some].cpu().numpy(), len(some), K) for w in (gate, up))
    x = torch.from_numpy(tokens(R, K)).to(cuda_dev)
    off = torch.zeros(E + 1, dtype=torch.int32, device=cuda_dev)
    off[E] = R
    h = gq_lib.mul_mat_grouped_swiglu(gate, up, t, E, M, K, x, off)[R - 20:][:, some]
    near(h, *gr.swiglu([wg], [wu], np.array([0, 20]), x[R - 20:].cpu().double().numpy(), np.zeros((20, len(some)))))


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
