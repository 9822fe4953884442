"""The experts of a layer as GGUF files hold them: 3-D tensors, uploaded and used as they are."""
import numpy as np
import pytest
import torch

import gguf_writer
import mx_reference as ref
from test_gpu_moe import random_blocks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,t_down", [("mxfp4", "mxfp4"), ("q4_k", "q8_0")])
def test_experts_of_a_file(gq_lib, cuda_dev, tmp_path, t, t_down):
    from block_quantized_matmul_gq_gb300 import gguf
    E, D, F = 3, 256, 512
    rng = np.random.default_rng(0)
    sizes = {"gate": (t, F, D), "up": (t, F, D), "down": (t_down, D, F)}
    blocks = {n: random_blocks(tt, E * rows, K, rng) for n, (tt, rows, K) in sizes.items()}
    raw, _ = gguf_writer.build([], [(n, (K, rows, E), gq_lib.TYPES[tt], blocks[n].tobytes())
                                    for n, (tt, rows, K) in sizes.items()])
    (tmp_path / "layer.gguf").write_bytes(raw)
    with gguf.GGUFFile(str(tmp_path / "layer.gguf")) as file:
        assert [i.shape for i in file.tensors()] == [(D, F, E), (D, F, E), (F, D, E)]
        gate, up, down = (file.upload(n, cuda_dev) for n in ("gate", "up", "down"))
    layer = gq_lib.MoeExperts(gate, up, down, t, E, D, F, t_down=t_down)
    x = rng.standard_normal((5, D)).astype(np.float32)
    ids = rng.integers(0, E, (5, 2)).astype(np.int32)
    w = rng.random((5, 2)).astype(np.float32)
    y = gq_lib.moe_swiglu(layer, *(torch.from_numpy(a).to(cuda_dev) for a in (x, ids, w)))
    cut = {n: [tuple(a[e * rows:(e + 1) * rows] for a in ref.weights(tt, blocks[n], E * rows, K)) for e in range(E)]
           for n, (tt, rows, K) in sizes.items()}
    want, tol = ref.moe(cut["gate"], cut["up"], cut["down"], x.astype(np.float64), ids, w)
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
