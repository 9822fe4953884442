"""The device checks of the MXFP4 and expert calls, with stand-ins for tensors of two GPUs: no
library function is reached with an address of another device than the current one."""
import pytest

torch = pytest.importorskip("torch")


class Tensor:
    """What the binding looks at of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = tuple(shape), dtype, index
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return self.index


class Library:
    """Counts the calls that arrive."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def binding(gq_lib, monkeypatch):
    monkeypatch.setattr(gq_lib, "lib", Library())
    monkeypatch.setattr(gq_lib, "_current_device", lambda: 0)
    monkeypatch.setattr(gq_lib, "_raw_stream", lambda dev: 0)
    return gq_lib


E, D, F, N, K = 2, 64, 32, 3, 2


def blocks(rows, k, index):
    return Tensor((rows, k // 32 * 17), torch.uint8, index)


def matrices(on):
    return blocks(E * F, D, on[0]), blocks(E * F, D, on[1]), blocks(E * D, F, on[2])


@pytest.mark.parametrize("on", [(0, 0, 1), (0, 1, 0), (1, 0, 0), (1, 1, 0)])
def test_experts_of_two_devices(binding, on):
    with pytest.raises(ValueError, match="one device"):
        binding.MoeExperts(*matrices(on), "mxfp4", E, D, F)


def moe(binding, experts=0, x=0, ids=0, weights=0, out=0, workspace=None):
    layer = binding.MoeExperts(*matrices((experts,) * 3), "mxfp4", E, D, F)
    ws = None if workspace is None else Tensor((1 << 20,), torch.uint8, workspace)
    return binding.moe_swiglu(layer, Tensor((N, D), torch.float32, x), Tensor((N, K), torch.int32, ids),
                              Tensor((N, K), torch.float32, weights), out=Tensor((N, D), torch.float32, out),
                              workspace=ws)


@pytest.mark.parametrize("where", ["experts", "x", "ids", "weights", "out", "workspace"])
def test_moe_on_another_device(binding, where):
    with pytest.raises(ValueError, match="cuda:1"):
        moe(binding, **{where: 1})
    if where != "workspace":
        with pytest.raises(ValueError, match="cuda:1"):
            moe(binding, **{where: 1, "workspace": 0})
    assert binding.lib.calls == []


def mx4x(binding, weights=0, x=0, out=0, workspace=None):
    ws = None if workspace is None else Tensor((1 << 20,), torch.uint8, workspace)
    return binding.mul_mat_mx4x(blocks(5, D, weights), "mxfp4", 5, D, Tensor((N, D), torch.float32, x),
                                out=Tensor((N, 5), torch.float32, out), workspace=ws)


@pytest.mark.parametrize("where", ["weights", "x", "out", "workspace"])
def test_mx4x_on_another_device(binding, where):
    with pytest.raises(ValueError, match="cuda:1"):
        mx4x(binding, **{where: 1})
    assert binding.lib.calls == []


def test_one_device_is_let_through(binding):
    moe(binding)
    moe(binding, workspace=0)
    mx4x(binding)
    mx4x(binding, workspace=0)
    assert binding.lib.calls == ["gq_moe_swiglu", "gq_moe_swiglu_ws", "gq_mul_mat_mx4x", "gq_mul_mat_mx4x_ws"]
