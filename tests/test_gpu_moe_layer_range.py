"""silu(gate) * up past the largest fp16 value: infinite in fp16, in its tokens alone; in bf16 an ordinary value."""
import pytest
import torch

import fp4_util as f4
import fp8_weight_only_amd as fw
from test_gpu_moe_layer import BF, DEV, FL, HF, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t", [1, 12, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_activations_stay_in_their_tokens(dtype, t, fmt):
    x, l, top, up, down, ub, db = make(t, fmt, t, 6, 2, 192, 128, dtype, FL, bias=True)
    ub[5, 17] = ub[5, 128 + 17] = 400.0  # h of place 17 is near 160000
    l[:, 5] = -20.0
    l[::3, 5] = 20.0
    large = torch.zeros(t, dtype=torch.bool, device=DEV)
    large[::3] = True
    out = fw.moe_layer(x, l, top, up, down, ub, db)
    if dtype == BF:
        ref, bound = reference(x, l, top, up, down, ub, db, True)
        f4.assert_within(out, ref, bound, "bf16")
        return
    assert torch.isfinite(out[~large]).all()
    w = f4.decode(*(p[5, :, :] for p in down), 128, dtype) if fmt == "fp4" else down[0][5].view(torch.float8_e4m3fn).double()
    assert not torch.isfinite(out[large]).any(), "an infinite h times any weight, zero among them, is not finite"
    zero = w[:, 17] == 0
    assert torch.isnan(out[large][:, zero]).all() and torch.isinf(out[large][:, ~zero]).all()
