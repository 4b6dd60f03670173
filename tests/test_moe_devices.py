"""Tensors on a GPU that is not the current one: every call goes to the tensors'
device. torch's default stream has the handle 0 on every GPU, so a launch from
another current device would go to that one's queue, in no order with the tensors'
own work. Stand-ins for the tensors and for the C entries; no GPU needed."""
import math

import pytest
import torch

import fp8_weight_only_amd as fw

BF, FL, I8, U8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.uint8, torch.int32
MOE = ("fp8w_route", "fp8w_linear_experts", "fp8w_combine", "fp8w_quantize_int8", "fp8w_quantize_activations_int8",
       "fp8w_gemm_int8", "fp8w_linear_int8")


class Tensor:
    """What the helpers ask of a contiguous tensor on cuda:1."""
    is_cuda = True
    device = torch.device("cuda:1")

    def __init__(self, *shape, dtype=FL):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 40

    def new_empty(self, shape, dtype=None):
        return Tensor(*shape, dtype=dtype or self.dtype)

    def reshape(self, *shape):
        return Tensor(*shape, dtype=self.dtype)

    view = reshape


class Gpus:
    """The current device, and the device that was current at each call of a C entry."""
    current = 0

    def __init__(self):
        self.calls = []

    def entry(self, name):
        def call(*args):
            self.calls.append((name, self.current))
            return fw.SUCCESS
        return call

    def guard(self):
        gpus = self

        class Device:
            def __init__(self, device):
                self.index = device if isinstance(device, int) else torch.device(device).index

            def __enter__(self):
                self.before, gpus.current = gpus.current, self.index

            def __exit__(self, *exc):
                gpus.current = self.before

        return Device


@pytest.fixture
def gpus(monkeypatch):
    g = Gpus()
    for name in MOE:
        monkeypatch.setattr(fw.moe, name, g.entry(name))
    monkeypatch.setattr(fw, "fp8w_quantize", g.entry("fp8w_quantize"))
    monkeypatch.setattr(fw, "_stream", lambda device: 0)
    monkeypatch.setattr(fw.moe, "_stream", lambda device: 0)
    monkeypatch.setattr(fw.moe, "_current_device", lambda: g.current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", g.guard())
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=FL, device=None: Tensor(*shape, dtype=dtype))
    return g


def _route_out(t, e, top):
    return fw.Route(Tensor(t, top), Tensor(t, top, dtype=I32), Tensor(e + 1, dtype=I32), Tensor(t * top, dtype=I32),
                    Tensor(t * top, dtype=I32))


CALLS = {
    "route into tensors": lambda: fw.route(Tensor(4, 16), 2, out=_route_out(4, 16, 2)),
    "route with a workspace": lambda: fw.route(Tensor(4, 16), 2, workspace=Tensor(64, dtype=U8)),
    "experts": lambda: fw.linear_experts(Tensor(8, 64, dtype=BF), Tensor(4, 32, 64, dtype=U8), Tensor(4, 32),
                                         Tensor(5, dtype=I32)),
    "experts with a workspace": lambda: fw.linear_experts(Tensor(8, 64, dtype=BF), Tensor(4, 32, 64, dtype=U8),
                                                          Tensor(4, 32), Tensor(5, dtype=I32),
                                                          workspace=Tensor(64, dtype=U8)),
    "combine": lambda: fw.combine(Tensor(8, 64, dtype=BF), Tensor(4, 2)),
    "int8 with a workspace": lambda: fw.linear_int8(Tensor(8, 64, dtype=BF), Tensor(32, 64, dtype=I8), Tensor(32),
                                                    workspace=Tensor(1 << 20, dtype=U8)),
    "int8 activations": lambda: fw.quantize_activations_int8(Tensor(8, 64, dtype=BF)),
    "int8 product": lambda: fw.gemm_int8(Tensor(8, 64, dtype=I8), Tensor(8), Tensor(32, 64, dtype=I8), Tensor(32)),
    "int8 weights": lambda: fw.quantize_int8(Tensor(32, 64)),
    "experts' weights": lambda: fw.quantize_experts(Tensor(4, 32, 64)),
}


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("call", CALLS)
def test_calls_go_to_the_tensors_device(gpus, call, current):
    gpus.current = current
    CALLS[call]()
    assert [device for _, device in gpus.calls] == [1], gpus.calls
    assert gpus.current == current
