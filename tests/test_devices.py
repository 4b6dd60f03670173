"""The FP8 layer's helpers with tensors on a GPU that is not the current one: every
call goes to the tensors' device. Stand-ins for the tensors and for the C entries;
no GPU needed."""
import pytest
import torch

import fp8_weight_only_amd as fw
from test_moe_devices import BF, U8, Gpus, Tensor

ENTRIES = ("fp8w_quantize", "fp8w_linear_with_path", "fp8w_linear_noalloc", "fp8w_dequantize_fallback",
           "fp8w_quantize_grouped", "fp8w_linear_grouped_with_workspace", "fp8w_dequantize_grouped",
           "fp8w_quantize_activations", "fp8w_gemm_w8a8", "fp8w_linear_w8a8", "fp8w_fnuz_to_ocp")
X, Q, S, G = (lambda: Tensor(8, 64, dtype=BF)), (lambda: Tensor(32, 64, dtype=U8)), (lambda: Tensor(32)), (
    lambda: Tensor(32, 2))

CALLS = {
    "quantize": lambda: fw.quantize(Tensor(32, 64)),
    "linear": lambda: fw.linear(X(), Q(), S()),
    "linear_noalloc": lambda: fw.linear_noalloc(X(), Q(), S()),
    "dequantize": lambda: fw.dequantize(Q(), S()),
    "quantize_grouped": lambda: fw.quantize_grouped(Tensor(32, 64), 32),
    "linear_grouped": lambda: fw.linear_grouped(X(), Q(), G()),
    "dequantize_grouped": lambda: fw.dequantize_grouped(Q(), G()),
    "quantize_activations": lambda: fw.quantize_activations(X()),
    "gemm_w8a8": lambda: fw.gemm_w8a8(Tensor(8, 64, dtype=U8), Tensor(8), Q(), S()),
    "linear_w8a8": lambda: fw.linear_w8a8(X(), Q(), S()),
    "fnuz_to_ocp": lambda: fw.fnuz_to_ocp(Q(), Q()),
}


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("call", CALLS)
def test_calls_go_to_the_tensors_device(monkeypatch, call, current):
    gpus = Gpus()
    gpus.current = current
    for name in ENTRIES:
        monkeypatch.setattr(fw, name, gpus.entry(name))
    monkeypatch.setattr(fw, "_stream", lambda device: 0)
    monkeypatch.setattr(fw.moe, "_current_device", lambda: gpus.current)
    monkeypatch.setattr(torch.cuda, "device", gpus.guard())
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=torch.float32, device=None: Tensor(*shape, dtype=dtype))
    CALLS[call]()
    assert [device for _, device in gpus.calls] == [1], gpus.calls
    assert gpus.current == current


def test_cpu_tensors_are_refused_as_before():
    x, q, s = torch.zeros((8, 64), dtype=BF), torch.zeros((32, 64), dtype=U8), torch.zeros(32)
    for call in (lambda: fw.quantize(torch.zeros(32, 64)), lambda: fw.linear(x, q, s), lambda: fw.dequantize(q, s),
                 lambda: fw.quantize_activations(x), lambda: fw.linear_w8a8(x, q, s), lambda: fw.fnuz_to_ocp(q),
                 lambda: fw.quantize_experts(torch.zeros(2, 32, 64))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
