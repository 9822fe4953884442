"""The adapters' workspace; no GPU."""
import ctypes

import pytest


@pytest.mark.parametrize("kind", [1, 30])
@pytest.mark.parametrize("r,K,M", [(8, 32, 32), (16, 4096, 4096), (24, 544, 100), (64, 4096, 11008), (256, 11008, 2048),
                                   (72, 16384, 70000), (8, 1 << 20, 8)])
def test_adapters_workspace_holds_smaller_batches(gq_lib, r, K, M, kind):
    """Never smaller for more tokens: a workspace for the largest batch is one for all."""
    a = gq_lib.Adapters(None, None, None, kind, 8, r, K, M)
    size = lambda n: gq_lib.lib.gq_lora_workspace_size(ctypes.byref(a), n)
    last = 0
    for n in list(range(1, 4500)) + [1 << i for i in range(13, 18)]:
        now = size(n)
        assert now >= last, (n, now, last)
        last = now
    assert size(4096) <= 4 * r * (16 * 912 + 2 * 4096)      # parts of K for all CTAs at most


def test_a_few_requests_need_little(gq_lib):
    a = gq_lib.Adapters(None, None, None, 1, 32, 16, 4096, 4096)
    assert gq_lib.lib.gq_lora_workspace_size(ctypes.byref(a), 64) <= 64 * 1024
