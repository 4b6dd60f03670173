"""Host-side checks of the 4-bit entry points (no GPU needed): invalid arguments are
refused before anything is enqueued, failed launches are raised once, calls go to the
tensors' GPU."""
import types

import pytest
import torch

import fp8_weight_only_amd as fw
from test_moe_abi import A, B, C, D, E, F, G, H
from test_moe_devices import BF, I32, U8, Tensor, gpus  # noqa: F401  (a fixture)


def _quantize(w=A, dtype=fw.BF16, n=8, k=70, q=B, s=C):
    return fw.fp8w_quantize_fp4(w, dtype, n, k, q, s, 0)


def test_quantize_refusals():
    for bad in [dict(dtype=3), dict(dtype=-1), dict(n=-1), dict(k=-1), dict(w=0), dict(q=0), dict(s=0), dict(q=A + 8 * 70),
                dict(s=A + 8 * 140 - 1), dict(s=B + 8 * 35 - 1), dict(n=1 << 31), dict(k=1 << 31)]:
        assert _quantize(**bad) == fw.ERR_INVALID_VALUE, bad
    assert _quantize(w=A + 1) == fw.ERR_MISALIGNED
    assert _quantize(w=A + 2, dtype=fw.FP32) == fw.ERR_MISALIGNED
    assert _quantize(n=0) == fw.SUCCESS and _quantize(k=0) == fw.SUCCESS


def _dequantize(q=A, s=B, n=8, k=70, out=C, dtype=fw.FP16):
    return fw.fp8w_dequantize_fp4(q, s, n, k, out, dtype, 0)


def test_dequantize_refusals():
    for bad in [dict(dtype=3), dict(n=-1), dict(k=-1), dict(q=0), dict(s=0), dict(out=0), dict(out=A), dict(out=B),
                dict(q=C + 8 * 140 - 1), dict(s=C + 8), dict(n=1 << 31)]:
        assert _dequantize(**bad) == fw.ERR_INVALID_VALUE, bad
    assert _dequantize(out=C + 1) == fw.ERR_MISALIGNED
    assert _dequantize(n=0) == fw.SUCCESS and _dequantize(k=0) == fw.SUCCESS


def _linear(x=A, act=fw.BF16, m=4, k=70, q=B, s=C, bias=D, n=8, y=E, ws=F, wsb=1 << 30):
    return fw.fp8w_linear_fp4(x, act, m, k, q, s, bias, n, y, ws, wsb, 0)


def test_linear_refusals():
    for bad in [dict(act=fw.FP32), dict(act=7), dict(m=-1), dict(k=-1), dict(n=-1), dict(x=0), dict(q=0), dict(s=0),
                dict(y=0), dict(y=A), dict(y=B + 8 * 35 - 2), dict(y=C + 8 * 3 - 2), dict(y=D + 14), dict(m=1 << 31),
                dict(n=1 << 31), dict(k=1 << 31), dict(m=1 << 30, n=1 << 20)]:
        assert _linear(**bad) == fw.ERR_INVALID_VALUE, bad
    for bad in [dict(x=A + 1), dict(bias=D + 1), dict(y=E + 1)]:
        assert _linear(**bad) == fw.ERR_MISALIGNED, bad
    assert _linear(m=0) == fw.SUCCESS and _linear(n=0) == fw.SUCCESS
    for sizes in [(0, 8, 70), (4, 0, 70), (-1, 8, 70), (4, 8, -1), (1 << 31, 8, 70)]:
        assert fw.fp8w_linear_fp4_kernel(*sizes, 0, 0, 0) is None
        assert fw.fp8w_linear_fp4_workspace_bytes(*sizes, 0, 0, 0) == 0
    assert fw.fp8w_linear_fp4_kernel(4, 8, 0, 0, 0, 0) is not None


@pytest.mark.parametrize("m,n,k", [(1, 4096, 14336), (22, 4096, 14336), (64, 1024, 8192), (200, 512, 8192),
                                   (500, 768, 14336), (40, 300, 8198), (4096, 14336, 4096)])
def test_linear_workspace_is_checked(m, n, k):
    need = fw.fp8w_linear_fp4_workspace_bytes(m, n, k, A, B, C)
    size = dict(m=m, n=n, k=k)
    if need:
        assert _linear(wsb=need - 1, **size) == fw.ERR_WORKSPACE
        assert _linear(ws=0, wsb=need, **size) == fw.ERR_WORKSPACE
        assert _linear(ws=F + 8, wsb=need, **size) == fw.ERR_MISALIGNED
        for other in (A, B, C, D, E):
            assert _linear(ws=other, wsb=need, **size) == fw.ERR_INVALID_VALUE


def _experts(x=A, act=fw.BF16, xc=8, k=256, q=B, s=C, bias=D, e=4, n=128, off=E, m=8, xr=F, yr=G, y=H):
    return fw.fp8w_linear_experts_fp4(x, act, xc, k, q, s, bias, e, n, off, m, xr, yr, y, 0)


def test_linear_experts_refusals():
    for bad in [dict(act=fw.FP32), dict(act=9), dict(xc=-1), dict(k=-1), dict(e=0), dict(e=1025), dict(n=-1),
                dict(m=-1), dict(xc=7, xr=0), dict(x=0), dict(q=0), dict(s=0), dict(off=0), dict(y=0), dict(y=A),
                dict(y=B + 4 * 128 * 128 - 2), dict(y=C + 4 * 128 * 8 - 2), dict(y=D), dict(y=E), dict(y=F), dict(y=G),
                dict(n=1 << 31), dict(m=1 << 31), dict(m=1 << 30, xc=1 << 30, n=1 << 20),
                dict(k=(1 << 31) - 1, n=(1 << 31) - 1)]:
        assert _experts(**bad) == fw.ERR_INVALID_VALUE, bad
    for bad in [dict(x=A + 1), dict(bias=D + 1), dict(off=E + 2), dict(xr=F + 2), dict(yr=G + 1), dict(y=H + 1)]:
        assert _experts(**bad) == fw.ERR_MISALIGNED, bad
    assert _experts(m=0, xc=0, xr=0) == fw.SUCCESS and _experts(n=0) == fw.SUCCESS
    assert fw.fp8w_linear_experts_fp4_kernel(0, 4, 128, 256, 0, 0, 0) is None
    assert fw.fp8w_linear_experts_fp4_kernel(8, 0, 128, 256, 0, 0, 0) is None


# ------------------------------------------------------------------ the helpers
FAST = {
    "linear_fp4": lambda t: fw.linear_fp4(t, t, t),
    "linear_experts_fp4": lambda t: fw.linear_experts_fp4(t, t, t, t),
}


@pytest.mark.parametrize("name", FAST)
def test_a_failed_launch_is_raised(name, monkeypatch):
    monkeypatch.setattr(fw.moe, "_FAST", types.SimpleNamespace(**{n: lambda *a: fw.ERR_HIP for n in FAST}))
    again = []
    monkeypatch.setattr(fw.moe, "fp8w_" + name, lambda *a: again.append(a) or fw.SUCCESS)
    with pytest.raises(fw.Fp8wMoeError) as err:
        FAST[name](torch.zeros(4, 8))
    assert err.value.status == fw.ERR_HIP and "fp8w_" + name in str(err.value) and not again


@pytest.mark.parametrize("name", FAST)
def test_a_refused_call_takes_the_python_path(name, monkeypatch):
    monkeypatch.setattr(fw.moe, "_FAST", types.SimpleNamespace(**{n: lambda *a: None for n in FAST}))
    with pytest.raises(ValueError, match="GPU tensor"):
        FAST[name](torch.zeros(4, 8))


def test_the_helpers_check_shapes_and_types():
    t = torch.zeros
    x = t(4, 70, dtype=BF)
    u = dict(dtype=U8)
    for call in [lambda: fw.quantize_fp4(t(4)), lambda: fw.quantize_fp4(t(4, 8)),
                 lambda: fw.dequantize_fp4(t(4, **u), t(4, **u)), lambda: fw.dequantize_fp4(t(4, 8, **u), t(4, 1, **u)),
                 lambda: fw.linear_fp4(x, t(8, 35, **u), t(8, 3, **u)), lambda: fw.linear_fp4(x[0], t(8, 35, **u), t(8, 3, **u)),
                 lambda: fw.linear_experts_fp4(x, t(2, 8, 35, **u), t(2, 8, 3, **u), t(3, dtype=I32))]:
        with pytest.raises(ValueError):
            call()


def _entries(gpus, monkeypatch):  # noqa: F811
    for name in ("fp8w_quantize_fp4", "fp8w_dequantize_fp4", "fp8w_linear_fp4", "fp8w_linear_experts_fp4"):
        monkeypatch.setattr(fw.moe, name, gpus.entry(name))


X, Q, S = Tensor(4, 70, dtype=BF), Tensor(8, 35, dtype=U8), Tensor(8, 3, dtype=U8)
CALLS = {
    "weights": lambda: fw.quantize_fp4(Tensor(8, 70)),
    "experts' weights": lambda: fw.quantize_fp4(Tensor(2, 8, 70)),
    "back": lambda: fw.dequantize_fp4(Q, S, 70),
    "linear with a workspace": lambda: fw.linear_fp4(X, Q, S, workspace=Tensor(1 << 20, dtype=U8)),
    "experts": lambda: fw.linear_experts_fp4(X, Tensor(2, 8, 35, dtype=U8), Tensor(2, 8, 3, dtype=U8),
                                             Tensor(3, dtype=I32)),
}


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("call", CALLS)
def test_calls_go_to_the_tensors_device(gpus, monkeypatch, call, current):  # noqa: F811
    _entries(gpus, monkeypatch)
    gpus.current = current
    CALLS[call]()
    assert [device for _, device in gpus.calls] == [1], gpus.calls
    assert gpus.current == current


@pytest.mark.parametrize("wrong", ["q", "s", "x type", "q type", "workspace device"])
def test_helpers_refuse_what_does_not_fit(gpus, monkeypatch, wrong):  # noqa: F811
    _entries(gpus, monkeypatch)
    x = Tensor(4, 70, dtype=torch.float32 if wrong == "x type" else BF)
    q = Tensor(8, 36 if wrong == "q" else 35, dtype=torch.int8 if wrong == "q type" else U8)
    s = Tensor(8, 2 if wrong == "s" else 3, dtype=U8)
    ws = torch.zeros(64) if wrong == "workspace device" else Tensor(64, dtype=U8)
    with pytest.raises((ValueError, TypeError)):
        fw.linear_fp4(x, q, s, workspace=ws)
    assert not gpus.calls
