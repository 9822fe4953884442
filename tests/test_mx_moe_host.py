"""MXFP4, router and expert-layer checks that need no GPU: sizes and refusals, before any CUDA
call; and the reference forms that the GPU tests use, against values worked out by hand."""
import ctypes

import numpy as np
import pytest

import mx_reference as ref

A16 = 0x7000_0000_0000
A8, A4, A2 = A16 + 8, A16 + 4, A16 + 2


def test_sizes(gq_lib):
    lib = gq_lib.lib
    assert gq_lib.TYPES["mxfp4"] == 39 and lib.gq_block_bytes(39) == 17
    assert lib.gq_row_bytes(39, 2048) == 64 * 17 and lib.gq_row_bytes(39, 40) == 0
    assert lib.gq_mul_mat_workspace_size(39, 64, 256, 0) == 0
    size = lib.gq_mul_mat_workspace_size
    for K, N in ((256, 3), (2048, 1), (32, 4096), (5632, 100)):
        n = N * (4 * K + K // 8)
        assert n < size(39, 64, K, N) <= n + 9 * 1024 and size(39, 64, K, N) % 256 == 0
    assert size(39, 64, 256, 5000) == size(39, 64, 256, 4096)
    assert lib.gq_mul_mat_mx4x_workspace_size(2, 64, 256, 3) == 0
    assert lib.gq_mul_mat_mx4x_workspace_size(39, 64, 256, 3) > 0


def test_mul_mat_refusals(gq_lib):
    lib = gq_lib.lib
    q = lib.gq_quantize_mxfp4
    assert q(A16, 4, 40, A16, None) == -2
    assert q(None, 4, 64, A16, None) == -1
    assert q(A2, 4, 64, A16, None) == -4
    assert q(A16, 4, 64, A8, None) == -4
    assert q(None, 0, 64, None, None) == 0
    assert lib.gq_dequantize(A8, 39, 4, 64, A16, None) == -4
    mm = lib.gq_mul_mat_ws
    assert mm(A16, 39, 4, 64, A16, 1, A16, None, 0, None) == -1            # workspace missing
    assert mm(A16, 39, 4, 64, A16, 1, A16, A16, 16, None) == -2            # and too small
    assert mm(A16, 39, 4, 64, A16, 1, A16, A16 + 16, 1 << 20, None) == -4  # and misaligned
    assert mm(A16, 39, 4, 40, A16, 1, A16, A16, 1 << 20, None) == -2
    assert lib.gq_mul_mat_q8x(A16, 39, 4, 256, A16, 1, A16, None) == -3
    assert lib.gq_mul_mat_q8x_batched(None, 0, 39, 1, None) == -3
    assert lib.gq_mul_mat_noalloc(A16, 39, 1, 1 << 25, A16, 1, A16, None) == -2   # token > 64 MiB
    mx = lib.gq_mul_mat_mx4x_ws
    assert mx(A16, 2, 4, 64, A16, 1, A16, A16, 1 << 20, None) == -3        # both operands MXFP4
    assert mx(A16, 39, 4, 40, A16, 1, A16, A16, 1 << 20, None) == -2
    assert mx(A8, 39, 4, 64, A16, 1, A16, A16, 1 << 20, None) == -4
    assert mx(A16, 39, 4, 64, A2, 1, A16, A16, 1 << 20, None) == -4
    assert mx(A16, 39, 4, 64, None, 1, A16, A16, 1 << 20, None) == -1
    assert mx(A16, 39, 4, 64, A16, 1, A16, None, 1 << 20, None) == -1
    assert mx(A16, 39, 4, 64, A16, 1, A16, A16, 8, None) == -2
    assert mx(A16, 39, 4, 64, A16, 1, A16, A16 + 128, 1 << 20, None) == -4
    assert mx(None, 39, 0, 64, None, 1, None, None, 0, None) == 0
    assert lib.gq_mul_mat_mx4x(None, 39, 4, 64, None, 0, None, None) == 0
    assert lib.gq_mul_mat_mx4x(A16, 12, 4, 256, A16, 1, A16, None) == -3


def test_route_refusals(gq_lib):
    r = gq_lib.lib.gq_moe_route
    assert r(A16, 1, 0, 1, 1, A16, A16, None) == -2
    assert r(A16, 1, 1025, 1, 1, A16, A16, None) == -2
    assert r(A16, 1, 8, 0, 1, A16, A16, None) == -2
    assert r(A16, 1, 8, 9, 1, A16, A16, None) == -2
    assert r(A16, 1, 128, 65, 1, A16, A16, None) == -2
    assert r(A16, -1, 8, 2, 1, A16, A16, None) == -2
    assert r(None, 1, 8, 2, 1, A16, A16, None) == -1
    assert r(A16, 1, 8, 2, 1, None, A16, None) == -1
    assert r(A16, 1, 8, 2, 1, A16, None, None) == -1
    assert r(A2, 1, 8, 2, 1, A16, A16, None) == -4
    assert r(None, 0, 8, 2, 1, None, None, None) == 0


def test_moe_refusals(gq_lib):
    lib, X = gq_lib.lib, gq_lib.Experts

    def call(N=1, k=2, x=A16, ids=A16, w=A16, y=A16, ws=A16, n=1 << 24, **over):
        a = dict(W_gate=A16, W_up=A16, W_down=A16, type=2, down_type=2, E=4, D=64, F=96)
        a.update(over)
        return lib.gq_moe_swiglu_ws(ctypes.byref(X(**a)), x, N, ids, w, k, y, ws, n, None)

    assert lib.gq_moe_swiglu(None, A16, 1, A16, A16, 1, A16, None) == -1
    assert call(type=7) == -3 and call(down_type=1) == -3
    assert call(E=0) == -2 and call(E=1025) == -2 and call(D=0) == -2 and call(F=0) == -2
    assert call(D=48) == -2 and call(F=40) == -2
    assert call(type=12) == -2 and call(down_type=12) == -2          # D = 64, F = 96 under Q4_K
    assert call(k=0) == -2 and call(k=65) == -2 and call(N=-1) == -2
    assert call(E=1024, F=1 << 22) == -2                             # E * F rows too many
    assert call(E=1, F=1 << 25) == -2 and call(E=1, D=1 << 25) == -2  # too wide
    for name in ("W_gate", "W_up", "W_down"):
        assert call(**{name: None}) == -1 and call(**{name: A8}) == -4
    for name in ("x", "ids", "w", "y"):
        assert call(**{name: None}) == -1 and call(**{name: A2}) == -4
    assert call(ws=None) == -1 and call(n=16) == -2 and call(ws=A16 + 16) == -4
    assert call(N=0, x=None, ids=None, w=None, y=None, ws=None) == 0
    good = X(A16, A16, A16, 2, 39, 4, 64, 96)
    assert lib.gq_moe_workspace_size(ctypes.byref(good), 3, 2) > 0
    assert lib.gq_moe_workspace_size(ctypes.byref(good), 0, 2) == 0
    assert lib.gq_moe_workspace_size(ctypes.byref(good), 3, 0) == 0
    assert lib.gq_moe_workspace_size(None, 3, 2) == 0


def test_binding_refusals(gq_lib):
    torch = pytest.importorskip("torch")
    b = torch.zeros((4, 34), dtype=torch.uint8)
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        gq_lib.mul_mat_mx4x(b, "mxfp4", 4, 64, x, out=torch.zeros(2, 4))
    with pytest.raises(ValueError):
        gq_lib.mul_mat_mx4x(b, "mxfp4", 5, 64, x)                    # too few blocks
    with pytest.raises(ValueError):
        gq_lib.mul_mat_mx4x(b, "mxfp4", 4, 64, torch.zeros(2, 32))
    with pytest.raises(ValueError):
        gq_lib.moe_route(torch.zeros(4), 2)
    with pytest.raises(ValueError, match="CUDA"):
        gq_lib.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        gq_lib.MoeExperts(b, b, b, "mxfp4", 4, 64, 64)


# ---- the reference forms ------------------------------------------------------------------

def test_reference_mx_by_hand():
    w = np.zeros((1, 32), np.float32)
    w[0, :9] = [6, 5, 3.5, 2.5, -1.25, 0.25, 0.26, -0.2, 7.9]      # largest 7.9: e = 0
    codes, scales = ref.mx_quantize(w)
    assert scales.tolist() == [[127]]
    assert codes[0, 0, :9].tolist() == [7, 6, 6, 4, 8 + 2, 0, 1, 8, 7]
    assert ref.mx_values(codes, scales)[0, :9].tolist() == [6, 4, 4, 2, -1, 0, 0.5, 0, 6]
    packed = ref.mx_pack(codes, scales)
    assert packed.shape == (1, 17) and packed[0, 0] == 127 and packed[0, 1] == 7
    back = ref.mx_unpack(packed)
    assert np.array_equal(back[0], codes) and np.array_equal(back[1], scales)


def test_reference_route_by_hand():
    z = np.array([[0.0, np.log(3.0), 0.0, -np.inf], [-np.inf] * 4], np.float32)
    ids, w = ref.route(z, 2, True)
    assert ids.tolist() == [[1, 0], [0, 1]]
    assert np.allclose(w, [[0.75, 0.25], [0, 0]])
    _, w = ref.route(z, 2, False)
    assert np.allclose(w[0], [0.6, 0.2])


def test_gguf_knows_mxfp4(gq_lib, tmp_path):
    pytest.importorskip("torch")
    import gguf_writer
    from block_quantized_matmul_gq_gb300 import gguf
    data = bytes(range(256))[:6 * 17]
    raw, _ = gguf_writer.build([], [("w", (64, 3), 39, data), ("experts", (32, 3, 2), 39, data)])
    path = tmp_path / "mx.gguf"
    path.write_bytes(raw)
    with gguf.GGUFFile(str(path)) as f:
        out = (ctypes.c_int(), ctypes.c_int64(), ctypes.c_int64())
        refs = [ctypes.byref(v) for v in out]
        assert gq_lib.lib.gq_gguf_tensor_matrix(f._h, 0, *refs) == 0
        assert [v.value for v in out] == [39, 3, 64]
        assert gq_lib.lib.gq_gguf_tensor_matrix(f._h, 1, *refs) == -2   # three dimensions
        info = gq_lib.GgufTensor()
        assert gq_lib.lib.gq_gguf_tensor_info(f._h, 1, ctypes.byref(info)) == 0
        assert info.nbytes == 6 * 17
        assert ctypes.string_at(gq_lib.lib.gq_gguf_tensor_data(f._h, 1), 102) == data
