"""Sizes of grouped products' workspaces, and which sizes are refused; no GPU."""
import pytest


def test_many_tokens_and_weight_rows(gq_lib):
    """N, E * M and R * M have ranges of their own; N * E * M is no size of anything."""
    size = gq_lib.lib.gq_mul_mat_grouped_workspace_size
    assert size(2, 1024, 1 << 20, 32, 2048) > 0
    assert size(8, 256, 2048, 2048, 1 << 22) > 0
    assert size(2, 1024, 1 << 20, 32, 1 << 21) == 0          # R * M
    # refused for its workspace, after the sizes: R rows out of many more tokens
    call = gq_lib.lib.gq_mul_mat_grouped_ws
    at = 0x7000_0000_0000
    assert call(at, 2, 256, 2048, 2048, at, 1 << 22, at, 8, at, 64, at, None, 0, None) == -1
    assert call(at, 2, 256, 2048, 2048, at, 1 << 30, at, 8, at, 64, at, None, 0, None) == -2      # N * K


@pytest.mark.parametrize("t", [2, 8, 12, 39])
def test_grouped_workspace_holds_smaller_batches(gq_lib, t):
    size = gq_lib.lib.gq_mul_mat_grouped_workspace_size
    last = 0
    for n in range(1, 3000):
        now = size(t, 60, 640, 1024, n)
        assert now >= last
        last = now
