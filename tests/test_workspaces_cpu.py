"""The gated layer's and the 4-bit weights' scratch, without a GPU: tensors that say they
are on a device, and a library that notes what it is called with."""
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from dense_gemm_accelerator_gb300 import gated, q4


class On(torch.Tensor):
    """A CPU tensor that names a CUDA device as its own."""
    number = 0

    @staticmethod
    def of(number, *shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(type(f"On{number}", (On,), {"number": number}))

    __torch_function__ = torch._C._disabled_torch_function_impl

    def get_device(self):
        return self.number

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.number)


class Library:
    """Sizes of 1000 bytes on device 0 and 5000 on device 1; each call's workspace."""

    def __init__(self):
        self.current, self.given = 0, []

    def size(self, *_):
        return (1000, 5000)[self.current]

    dga_gated_workspace_size = dga_gated_backward_workspace_size = size
    dga_q4_linear_workspace_size = dga_q4_gated_workspace_size = size

    def call(self, *args):  # ..., workspace, its bytes, stream
        self.given.append(args[-2])
        return 0

    dga_gated = dga_gated_backward = dga_q4_linear = dga_q4_gated = call


@pytest.fixture
def fake(monkeypatch):
    library, empty = Library(), torch.empty
    for module in (gated, q4):
        monkeypatch.setattr(module, "lib", lambda: library)
        monkeypatch.setattr(module, "_raw_stream", lambda d: 0)
        monkeypatch.setattr(module, "_current_device", lambda: library.current)
        monkeypatch.setattr(module, "_elsewhere", lambda d: False)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    sizes = (gated._forward_workspace, gated._backward_workspace, q4._linear_workspace, q4._gated_workspace)
    for size in sizes:
        size.cache_clear()
    yield library
    for size in sizes:
        size.cache_clear()


def _calls(d, workspace=None):
    """Every call that takes a workspace, on device d, of one shape."""
    X, W, P, G = (On.of(d, *s) for s in ((40, 16), (48, 16), (40, 48), (40, 24)))
    Xh = On.of(d, 40, 20, dtype=torch.bfloat16)
    Q = dga.Q4Tensor(20, 32, On.of(d, 48, 16, dtype=torch.uint8), On.of(d, 48, 1, dtype=torch.bfloat16))
    yield lambda: dga.gated_forward(X, W, workspace=workspace)
    yield lambda: dga.gated_backward(X, W, P, G, workspace=workspace)
    yield lambda: dga.q4_linear_forward(Xh, Q, workspace=workspace)
    yield lambda: dga.q4_gated_forward(Xh, Q, workspace=workspace)


def test_each_device_has_its_own_size(fake):
    for d, size in ((0, 1000), (1, 5000), (0, 1000)):
        fake.current = d
        for call in _calls(d):
            call()
        assert fake.given == [size] * 4, d
        fake.given.clear()


def test_workspaces_that_are_refused(fake):
    """One on the host, on another device, or whose values are not all its own."""
    whole = On.of(0, 4096, dtype=torch.uint8)
    for bad in (torch.zeros(4096, dtype=torch.uint8), On.of(1, 4096, dtype=torch.uint8), On.of(0, 1, dtype=torch.uint8).expand(4096), whole[::2]):
        for call in _calls(0, bad):
            with pytest.raises(ValueError):
                call()
    assert not fake.given
    for call in _calls(0, whole):
        call()
    assert fake.given == [4096] * 4
