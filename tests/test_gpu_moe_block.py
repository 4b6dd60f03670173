"""The mixture-of-experts block of examples/moe_block.py against its 64-bit form,
and the operators where offsets pass 32 bits."""
import os
import sys

import pytest
import torch

import fp8_weight_only_amd as fw

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("t,hidden,inner,experts,top,dtype", [(1, 512, 256, 8, 2, BF), (1, 1024, 320, 64, 8, HF),
                                                             (37, 640, 448, 16, 4, BF), (300, 333, 129, 5, 3, HF),
                                                             (1500, 512, 256, 8, 2, BF)])
def test_block(t, hidden, inner, experts, top, dtype):
    block = moe_block.build(hidden, inner, experts, top, seed=t)
    x = torch.randn((t, hidden), generator=torch.Generator(device="cuda").manual_seed(t), device="cuda").to(dtype)
    out, r = block(x)
    want, bound = moe_block.reference(block, x, r)
    assert ((out.double() - want).abs() <= bound).all()


def test_experts_codes_past_32_bits():
    """4.4 GB of codes; the last expert's are read."""
    e, n, k, m = 75, 14336, 4096, 40
    q = torch.zeros((e, n, k), dtype=torch.uint8, device="cuda")
    q[-1] = torch.randint(0, 120, (n, k), dtype=torch.uint8, device="cuda")
    s = torch.full((e, n), 2.0 ** -9, device="cuda")
    offsets = torch.full((e + 1,), 0, dtype=torch.int32, device="cuda")
    offsets[-1] = m
    x = torch.randn((m, k), device="cuda").to(BF)
    w = (moe_block._e4m3(q[-1]) * 2.0 ** -9).t().contiguous()
    ref, mag = torch.mm(x.double(), w), torch.mm(x.double().abs(), w.abs())
    tol = ref.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + mag * (k + 8) * 2.0 ** -23
    for rows in (m, 1):  # a tile of rows, and one token
        offsets[-1] = rows
        y = fw.linear_experts(x[:rows].contiguous(), q, s, offsets).double()
        assert ((y - ref[:rows]).abs() <= tol[:rows]).all()


def test_gathered_rows_past_32_bits():
    """2.7 GB of activations; rows from its end are gathered."""
    rows, k, n, m = 330000, 4096, 256, 200
    x = torch.zeros((rows, k), dtype=BF, device="cuda")
    x[-m:] = torch.randn((m, k), device="cuda").to(BF)
    q, s = fw.quantize_experts(torch.randn((2, n, k), device="cuda") * 0.02)
    at = (rows - 1 - torch.arange(m, device="cuda")).int()
    offsets = torch.tensor([0, 50, m], dtype=torch.int32, device="cuda")
    y = fw.linear_experts(x, q, s, offsets, x_rows=at).double()
    for i, (lo, hi) in enumerate(((0, 50), (50, m))):
        w = (moe_block._e4m3(q[i]) * s[i].double()[:, None]).t().contiguous()
        xi = x[at[lo:hi].long()].double()
        ref, mag = torch.mm(xi, w), torch.mm(xi.abs(), w.abs())
        tol = ref.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + mag * (k + 8) * 2.0 ** -23
        assert ((y[lo:hi] - ref).abs() <= tol).all()


def test_outputs_past_32_bits():
    """Sums over 2.3 billion values, and an int8 layer with as many outputs: the last rows."""
    t, top, n = 70000, 8, 4096
    y = torch.zeros((t * top, n), dtype=BF, device="cuda")
    y[-top:] = 1.0
    w = torch.full((t, top), 0.25, device="cuda")
    out = fw.combine(y, w)
    assert (out[-1] == 2).all() and (out[:-1] == 0).all()
    del y, out
    m, n, k = 160000, 14400, 64
    x = torch.zeros((m, k), dtype=BF, device="cuda")
    x[-1] = 1.0
    q = torch.ones((n, k), dtype=torch.int8, device="cuda")
    out = fw.linear_int8(x, q, torch.full((n,), 0.5, device="cuda"))
    # 64 codes of 127 at scale 1 / 127 (fp32): within a rounding of 32
    assert ((out[-1].double() - 32).abs() <= 32 * 2.0 ** -8).all() and (out[-2] == 0).all()
