"""A feed-forward block on 4-bit weights as a serving program runs it: a prompt through the
experts' products, then single steps through the whole-layer call inside one captured graph,
a dense projection before and a shared expert beside it, against 64 bits.
"""
import pytest
import torch

import fp4_util as f4
import fp8_weight_only_amd as fw
from test_gpu_moe_layer import make, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


def _block(dtype, hidden=256, inner=192, e=12, top=3):
    x, l, top, up, down, ub, db = make(11, "fp4", 64, e, top, hidden, inner, dtype, bias=True)
    g = torch.Generator(device=DEV).manual_seed(12)
    proj = fw.quantize_fp4(torch.randn((hidden, hidden), generator=g, device=DEV) / hidden ** 0.5)
    shared = fw.quantize_fp4(torch.randn((hidden, hidden), generator=g, device=DEV) / hidden ** 0.5)
    router = torch.randn((hidden, e), generator=g, device=DEV)
    return x, router, top, up, down, ub, db, proj, shared


def _prompt(x, b):
    _, router, top, up, down, ub, db, proj, shared = b
    h = fw.linear_fp4(x, *proj)
    l = h.float() @ router
    r = fw.route(l, top)
    g = fw.linear_experts_fp4(h, *up, r.offsets, ub, x_rows=r.tokens)
    n = up[0].shape[1] // 2
    a = (torch.nn.functional.silu(g[:, :n].float()) * g[:, n:].float()).to(x.dtype)
    y = fw.combine(fw.linear_experts_fp4(a, *down, r.offsets, db, y_rows=r.slots), r.weights)
    return h, l, y, fw.linear_fp4(h, *shared)


def _step(x, b, l, out):
    _, router, top, up, down, ub, db, proj, shared = b
    h = fw.linear_fp4(x, *proj)
    y = fw.moe_layer(h, l, top, up, down, ub, db)
    out.copy_(y + fw.linear_fp4(h, *shared))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_prompt_and_its_steps(dtype):
    b = _block(dtype)
    x, top, up, down, ub, db, proj, shared = b[0], *b[2:]
    k = x.shape[1]
    h, l, y, z = _prompt(x, b)
    ref, mag = f4.product(x, f4.decode(*proj, k, dtype), None)
    f4.assert_within(h, ref, f4.tolerance(ref, mag, k, dtype), "projection")
    ref, mag = f4.product(h, f4.decode(*shared, k, dtype), None)
    f4.assert_within(z, ref, f4.tolerance(ref, mag, k, dtype), "shared expert")
    ref, bound = reference(h, l, top, up, down, ub, db, True)
    assert ((y.double() - ref).norm() / ref.norm()).item() < 4 * f4.half_step(dtype)
    f4.assert_within(fw.moe_layer(h, l, top, up, down, ub, db), ref, bound, "layer")
    # the same tokens one and eight at a time, in graphs
    for t in (1, 8):
        xs, ls, out = x[:t].clone(), l[:t].clone(), torch.empty((t, k), dtype=dtype, device=DEV)
        _step(xs, b, ls, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _step(xs, b, ls, out)
        for at in range(0, 32, t):
            xs.copy_(x[at:at + t])
            ls.copy_(l[at:at + t])
            graph.replay()
            hs = fw.linear_fp4(xs, *proj)
            want = fw.moe_layer(hs, ls, top, up, down, ub, db) + fw.linear_fp4(hs, *shared)
            torch.cuda.synchronize()
            assert torch.equal(out, want), at
            r64, limit = reference(hs, ls, top, up, down, ub, db, True)
            zs, ms = f4.product(hs, f4.decode(*shared, k, dtype), None)
            total = r64 + zs  # each part rounded, and their sum
            f4.assert_within(out, total, limit + f4.tolerance(zs, ms, k, dtype) +
                             (total.abs() + limit) * 1.01 * f4.half_step(dtype) + f4.tiny(dtype), f"step {at}")
