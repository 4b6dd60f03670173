"""A call whose launch failed in the compiled helpers is raised: not given to the
Python path, which would enqueue it again. A stand-in for the helpers; no GPU
needed."""
import types

import pytest
import torch

import fp8_weight_only_amd as fw

CALLS = {
    "route": lambda t: fw.route(t, 2),
    "linear_experts": lambda t: fw.linear_experts(t, t, t, t),
    "combine": lambda t: fw.combine(t, t),
    "linear_int8": lambda t: fw.linear_int8(t, t, t),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_raised(name, monkeypatch):
    helpers = types.SimpleNamespace(**{n: lambda *a: fw.ERR_HIP for n in CALLS})
    monkeypatch.setattr(fw.moe, "_FAST", helpers)
    again = []
    monkeypatch.setattr(fw.moe, "fp8w_" + name, lambda *a: again.append(a) or fw.SUCCESS)
    with pytest.raises(fw.Fp8wMoeError) as err:
        CALLS[name](torch.zeros(4, 8))
    assert err.value.status == fw.ERR_HIP and "fp8w_" + name in str(err.value) and not again


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_call_takes_the_python_path(name, monkeypatch):
    """None: the arguments' checks say what is wrong."""
    monkeypatch.setattr(fw.moe, "_FAST", types.SimpleNamespace(**{n: lambda *a: None for n in CALLS}))
    with pytest.raises(ValueError, match="GPU tensor"):
        CALLS[name](torch.zeros(4, 8))
