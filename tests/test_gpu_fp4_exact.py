"""The products on 4-bit weights and the whole layer on inputs whose sums are exact (exact_util): every result is known
bit for bit, so a block of k that is lost or taken twice, sums joined in fewer bits, or a slice that is read before it is
written shows however long the rows are, where the tolerances of the other tests grow with k. Workspaces are filled with
NaN and end in guard bytes.

The layer: logits are equal where they are finite, so weights are 1 / top_k, a power of two. Gates are whole numbers from
18 on, where 1 + exp(-g) rounds to 1 and silu(g) is g; up products are small whole numbers, so silu(g) * u is exact in
fp32 and its one rounding to the activation type is known. Down products and their weighted sum are exact.
"""
import pytest
import torch

import exact_util as ex
import fp4_util as f4
import fp8_weight_only_amd as fw
from test_gpu_fp4_plans import EXPERTS, LINEAR
from test_gpu_moe_layer_plans import ROWS, SHARED

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


def _workspace(need):
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)
    return ws, ws[:need]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,kernel", LINEAR)
def test_linear(m, n, k, kernel, dtype):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = ex.whole((m, k), g, dtype)
    q, s = ex.fp4_weights((n, k), g)
    b = ex.whole((n,), g, dtype, 60) if dtype == HF else None
    ws, part = _workspace(fw.fp4_workspace_bytes(x, q, s))
    out = torch.full((m + 2, n), float("nan"), dtype=dtype, device=DEV)
    fw.linear_fp4(x, q, s, b, out=out[1:-1], workspace=part if part.numel() else None)
    ex.assert_bits(out[1:-1], ex.product(x, f4.decode(q, s, k, dtype), b), kernel)
    assert (ws[part.numel():] == 0xff).all(), "wrote outside the workspace"
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all(), "wrote outside the output"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts(m, e, n, k, kernel, dtype):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = ex.whole((m, k), g, dtype)
    q, s = ex.fp4_weights((e, n, k), g)
    b = ex.whole((e, n), g, dtype, 60) if dtype == HF else None
    ends = torch.sort(torch.randint(0, m + 1, (e,), generator=g, device=DEV)).values.tolist()
    offsets = torch.tensor([0] + ends, dtype=torch.int32, device=DEV)
    xi = torch.randint(0, m, (m,), generator=g, device=DEV).int()
    yi = torch.randperm(m, generator=g, device=DEV).int()
    out = torch.full((m, n), float("nan"), dtype=dtype, device=DEV)
    fw.linear_experts_fp4(x, q, s, offsets, b, x_rows=xi, y_rows=yi, out=out)
    ref = torch.zeros((m, n), dtype=torch.float64, device=DEV)
    for i, lo, hi in zip(range(e), [0] + ends, ends):
        if hi > lo:
            ref[yi[lo:hi].long()] = ex.product(x[xi[lo:hi].long()], f4.decode(q[i], s[i], k, dtype),
                                               None if b is None else b[i])
    ex.assert_bits(out, ref, kernel)


def _stack(fmt, e, n, k, nonzero, g):
    """(q, scale) and the weights [e, n, k] in fp64: 1 and -1 in `nonzero` of the places, times 1 or 2."""
    at = torch.rand((e, n, k), generator=g, device=DEV)
    w = torch.where(at < nonzero, torch.where(at < nonzero / 2, 1.0, -1.0), 0.0)
    if fmt == "e4m3":
        scale = torch.randint(1, 3, (e, n), generator=g, device=DEV).float()
        return (w.to(torch.float8_e4m3fn).view(torch.uint8), scale), w.double() * scale.double()[:, :, None]
    code = torch.where(w > 0, 2, torch.where(w < 0, 10, 0)).to(torch.uint8)  # 1.0, -1.0, 0
    code = torch.nn.functional.pad(code, (0, k % 2))
    scale = torch.randint(127, 129, (e, n, (k + 31) // 32), generator=g, device=DEV, dtype=torch.uint8)
    by = torch.pow(2.0, scale.double() - 127).repeat_interleave(32, dim=2)[:, :, :k]
    return (code[:, :, 0::2] | (code[:, :, 1::2] << 4), scale), w.double() * by


def _layer(seed, fmt, t, e, top, hidden, inner, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = ex.whole((t, hidden), g, dtype, 1)
    # about eight terms of 1 or 2 to a gate or up product, around a gate of 70
    up, wu = _stack(fmt, e, 2 * inner, hidden, min(1.0, 12.0 / hidden), g)
    down, wd = _stack(fmt, e, hidden, inner, min(0.5, (300.0 if top == 64 else 1000.0) / inner), g)
    ub, db = ex.whole((e, 2 * inner), g, dtype, 3), ex.whole((e, hidden), g, dtype, 60)
    ub[:, :inner] += 70
    order = torch.rand((t, e), generator=g, device=DEV).argsort(dim=1)
    l = torch.where(order < top, 0.5, float("-inf"))
    if t > 4:
        l[4::9] = float("-inf")
    ws, part = _workspace(fw.moe_layer_workspace_bytes(x, l, top, up))
    out = torch.full((t + 2, hidden), float("nan"), dtype=dtype, device=DEV)
    fw.moe_layer(x, l, top, up, down, ub, db, renormalize=seed % 2 == 0, out=out[1:-1], workspace=part)
    ref = torch.zeros((t, hidden), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    for i in range(e):
        tok = (l[:, i] == 0.5).nonzero()[:, 0]
        if not tok.numel():
            continue
        r = ex.product(x[tok], wu[i], ub[i])
        gate, lift = r[:, :inner], r[:, inner:]
        assert gate.min().item() >= 18 and (gate * lift).abs().max().item() < 60000
        h = (gate * lift).float().to(dtype)
        ref[tok] += ex.product(h, wd[i], db[i]) / top
        mag[tok] += (torch.mm(h.double().abs(), wd[i].abs().t().contiguous()) + db[i].double().abs()) / top
    assert mag.max().item() < ex.BITS / top
    ex.assert_bits(out[1:-1], ref, f"{fmt} t={t} e={e} top={top} hidden={hidden} inner={inner}")
    assert (ws[part.numel():] == 0xff).all(), "wrote outside the workspace"
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all(), "wrote outside the output"


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t", [1, 16, 33, 64])
@pytest.mark.parametrize("hidden,inner", ROWS)
def test_layer(hidden, inner, t, fmt):
    _layer(t + hidden, fmt, t, 8, 4, hidden, inner, HF if (t + inner) % 2 else BF)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t,e,top,hidden,inner", SHARED)
def test_layer_shared_steps(t, e, top, hidden, inner, fmt, dtype):
    _layer(t + e, fmt, t, e, {3: 2}.get(top, top), hidden, inner, dtype)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t,e,top,hidden,inner", [(1, 8, 2, 4096, 3584), (64, 8, 8, 1024, 512), (16, 128, 8, 1024, 256),
                                                  (40, 2, 1, 512, 2048), (5, 1, 1, 256, 8200)])
def test_layer_sizes(t, e, top, hidden, inner, fmt):
    _layer(t, fmt, t, e, top, hidden, inner, BF)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t,e,top,hidden,inner", [(2, 1, 1, 1 << 22, 24), (1, 1, 1, (1 << 22) - 1, 9), (2, 1, 1, 24, 1 << 22),
                                                  (17, 1, 1, 9, (1 << 22) - 3), (64, 64, 64, 17, 32700), (64, 1024, 2, 40, 96)])
def test_layer_largest_widths(t, e, top, hidden, inner, fmt):
    """The longest rows of either launch, and the most values between them."""
    _layer(t, fmt, t, e, top, hidden, inner, BF)


LONG = [(1, 48, 1 << 22), (3, 40, (1 << 22) - 2), (3, 40, (1 << 22) + 2), (20, 40, (1 << 22) + 128), (2, 16, 5000001)]


@pytest.mark.parametrize("m,n,k", LONG)
def test_linear_longest_rows(m, n, k):
    """Up to the stream's and the rings' longest rows, and past them."""
    g = torch.Generator(device=DEV).manual_seed(k)
    x = ex.whole((m, k), g, BF, 1)
    (q, s), w = _stack("fp4", 1, n, k, 0.5, g)
    ex.assert_bits(fw.linear_fp4(x, q[0], s[0]), ex.product(x, w[0], unit=1.0), f"{m} {n} {k}")


@pytest.mark.parametrize("m,e,n,k", [(300, 1024, 64, 256), (300, 1024, 70, 101), (3000, 1024, 64, 256), (40, 2, 64, (1 << 22) + 2)])
def test_experts_largest(m, e, n, k):
    """The most experts, most of them empty; the longest rows."""
    g = torch.Generator(device=DEV).manual_seed(m + k)
    x = ex.whole((m, k), g, BF, 1)
    (q, s), w = _stack("fp4", e, n, k, 0.5, g)
    ids = torch.sort(torch.randint(0, e, (m,), generator=g, device=DEV)).values
    offsets = torch.searchsorted(ids, torch.arange(e + 1, device=DEV)).int()
    out = fw.linear_experts_fp4(x, q, s, offsets)
    ref = torch.cat([ex.product(x[ids == i], w[i], unit=1.0) for i in torch.unique(ids).tolist()])
    ex.assert_bits(out, ref, f"{m} {e} {n} {k}")
