"""Host-side checks of the whole mixture-of-experts layer (no GPU needed): invalid
arguments are refused before anything is enqueued, the workspace is checked, failed
launches are raised once, calls go to the tensors' GPU."""
import types

import pytest
import torch

import fp8_weight_only_amd as fw
from test_moe_devices import BF, U8, Tensor, gpus  # noqa: F401  (a fixture)

FL = torch.float32
STEP = 1 << 28
X, L, QU, SU, BU, QD, SD, BD, OUT, WS = (STEP * i for i in range(1, 11))


def _layer(x=X, act=fw.BF16, t=4, hidden=64, l=L, lt=fw.FP32, e=8, top=2, renorm=1, fmt=fw.WEIGHT_FP4, qu=QU, su=SU, bu=BU,
           inner=40, qd=QD, sd=SD, bd=BD, out=OUT, ws=WS, wsb=1 << 27):
    return fw.fp8w_moe_layer(x, act, t, hidden, l, lt, e, top, renorm, fmt, qu, su, bu, inner, qd, sd, bd, out, ws, wsb, 0)


@pytest.mark.parametrize("fmt", [fw.WEIGHT_E4M3, fw.WEIGHT_FP4])
def test_layer_refusals(fmt):
    for bad in [dict(act=fw.FP32), dict(act=7), dict(lt=5), dict(t=-1), dict(t=65), dict(e=0), dict(e=1025), dict(top=0),
                dict(top=9), dict(e=256, top=65), dict(hidden=0), dict(inner=0), dict(hidden=-1), dict(inner=-4),
                dict(hidden=(1 << 22) + 1), dict(inner=(1 << 22) + 1), dict(t=64, top=8, inner=1 << 19), dict(x=0), dict(l=0),
                dict(qu=0), dict(su=0), dict(qd=0), dict(sd=0), dict(out=0)]:
        assert _layer(fmt=fmt, **bad) == fw.ERR_INVALID_VALUE, bad
    assert _layer(fmt=7) == fw.ERR_INVALID_VALUE
    for at in (X, L, QU, SU, BU, QD, SD, BD):  # neither the result nor the workspace on an input
        assert _layer(fmt=fmt, out=at) == fw.ERR_INVALID_VALUE, at
        assert _layer(fmt=fmt, ws=at) == fw.ERR_INVALID_VALUE, at
    assert _layer(fmt=fmt, out=WS + 64) == fw.ERR_INVALID_VALUE
    for bad in [dict(x=X + 1), dict(l=L + 2), dict(bu=BU + 1), dict(bd=BD + 1), dict(out=OUT + 1), dict(ws=WS + 8)]:
        assert _layer(fmt=fmt, **bad) == fw.ERR_MISALIGNED, bad
    assert _layer(fmt=fmt, t=0) == fw.SUCCESS
    assert _layer(fmt=fw.WEIGHT_E4M3, su=SU + 2) == fw.ERR_MISALIGNED
    assert _layer(fmt=fw.WEIGHT_E4M3, sd=SD + 1) == fw.ERR_MISALIGNED


@pytest.mark.parametrize("t,e,top,hidden,inner", [(1, 8, 2, 4096, 14336), (64, 8, 2, 4096, 14336), (13, 60, 4, 1030, 513),
                                                  (16, 128, 8, 64, 2000), (64, 1024, 64, 1, 1)])
def test_layer_workspace_is_checked(t, e, top, hidden, inner):
    need = fw.fp8w_moe_layer_workspace_bytes(t, e, top, hidden, inner)
    assert need >= 2 * t * top * inner
    sizes = dict(t=t, e=e, top=top, hidden=hidden, inner=inner)
    # addresses too far apart for these sizes to meet
    far = dict(zip(("x", "l", "qu", "su", "bu", "qd", "sd", "bd", "out", "ws"), ((1 << 40) * i for i in range(1, 11))))
    assert _layer(**sizes, **far, wsb=need - 1) == fw.ERR_WORKSPACE
    assert _layer(**sizes, **dict(far, ws=0), wsb=need) == fw.ERR_WORKSPACE
    assert _layer(**sizes, **dict(far, ws=far["ws"] + 4), wsb=need) == fw.ERR_MISALIGNED


def test_layer_workspace_of_invalid_sizes():
    for sizes in [(0, 8, 2, 64, 32), (65, 8, 2, 64, 32), (4, 0, 2, 64, 32), (4, 8, 9, 64, 32), (4, 8, 2, 0, 32),
                  (4, 8, 2, 64, 0), (4, 8, 2, 1 << 23, 32)]:
        assert fw.fp8w_moe_layer_workspace_bytes(*sizes) == 0, sizes


def _tensors(**other):
    t = dict(x=Tensor(4, 64, dtype=BF), logits=Tensor(4, 8, dtype=FL), qu=Tensor(8, 80, 32, dtype=U8),
             su=Tensor(8, 80, 2, dtype=U8), qd=Tensor(8, 64, 20, dtype=U8), sd=Tensor(8, 64, 2, dtype=U8), ws=None, top=2)
    t.update(other)
    return lambda: fw.moe_layer(t["x"], t["logits"], t["top"], (t["qu"], t["su"]), (t["qd"], t["sd"]), workspace=t["ws"])


@pytest.mark.parametrize("current", [0, 1])
def test_calls_go_to_the_tensors_device(gpus, monkeypatch, current):  # noqa: F811
    monkeypatch.setattr(fw.moe, "fp8w_moe_layer", gpus.entry("fp8w_moe_layer"))
    gpus.current = current
    _tensors(ws=Tensor(1 << 20, dtype=U8))()
    assert [device for _, device in gpus.calls] == [1], gpus.calls
    assert gpus.current == current


@pytest.mark.parametrize("wrong", [dict(x=Tensor(4, 64, dtype=FL)), dict(x=Tensor(4, 65, dtype=BF)),
                                   dict(logits=Tensor(5, 8, dtype=FL)), dict(logits=Tensor(4, 9, dtype=FL)),
                                   dict(qu=Tensor(8, 81, 32, dtype=U8), su=Tensor(8, 81, 2, dtype=U8)),
                                   dict(su=Tensor(8, 80, 3, dtype=U8)), dict(qd=Tensor(8, 64, 21, dtype=U8)),
                                   dict(sd=Tensor(8, 63, 2, dtype=U8)), dict(qd=Tensor(8, 64, 40, dtype=U8),
                                                                            sd=Tensor(8, 64, dtype=FL)),
                                   dict(ws=torch.zeros(64)), dict(top=0), dict(top=9)])
def test_layer_refuses_what_does_not_fit(gpus, monkeypatch, wrong):  # noqa: F811
    monkeypatch.setattr(fw.moe, "fp8w_moe_layer", gpus.entry("fp8w_moe_layer"))
    with pytest.raises((ValueError, TypeError)):
        _tensors(**wrong)()
    assert not gpus.calls


def test_a_failed_launch_is_raised(monkeypatch):
    monkeypatch.setattr(fw.moe, "_FAST", types.SimpleNamespace(moe_layer=lambda *a: fw.ERR_HIP))
    again = []
    monkeypatch.setattr(fw.moe, "fp8w_moe_layer", lambda *a: again.append(a) or fw.SUCCESS)
    t = torch.zeros(4, 8)
    with pytest.raises(fw.Fp8wMoeError) as err:
        fw.moe_layer(t, t, 2, (t, t), (t, t))
    assert err.value.status == fw.ERR_HIP and "fp8w_moe_layer" in str(err.value) and not again


def test_a_refused_call_takes_the_python_path(monkeypatch):
    monkeypatch.setattr(fw.moe, "_FAST", types.SimpleNamespace(moe_layer=lambda *a: None))
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        fw.moe_layer(t, t, 2, (t, t), (t, t))
