"""A workspace for the largest batch serves every smaller one."""
import pytest
import torch

from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r,K,M,largest", [(16, 4096, 4096, 2081), (64, 2048, 512, 961), (8, 8192, 64, 3000)])
def test_one_workspace(gq_lib, cuda_dev, r, K, M, largest):
    c = Case(gq_lib, cuda_dev, torch.float16, 3, r, K, M, largest)
    n = c.adapters.workspace_size(largest)
    around = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=cuda_dev)
    for N in (1, 5, 39, 152, 600, 912, 960, 2080, largest):
        if N > largest:
            continue
        args = (c.adapters, c.X[:N], c.ids[:N], c.Y[:N])
        assert torch.equal(gq_lib.lora_add(*args, workspace=around[256:256 + n]), gq_lib.lora_add(*args))
    assert (around[:256] == 0xA5).all() and (around[256 + n:] == 0xA5).all()
