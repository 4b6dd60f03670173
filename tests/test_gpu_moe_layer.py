"""GPU parity of the whole mixture-of-experts layer against a 64-bit computation
that makes its own choice of experts.

The tolerance follows the roundings: the fp32 sums of both products (2^-23 of the
magnitudes summed, per product), the activation (a slope below 1.1, its own few fp32
steps), the rounding of silu(gate) * up to the activation type, the router's weight
(as in the router's own test), the weighted sum, and the rounding of the result.
"""
import pytest
import torch

import fp4_util as f4
import fp8_weight_only_amd as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
EPS = 2.0 ** -23


def _e4m3(q, s):
    c = q.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(c >= 128, -mag, mag) * s.double()[:, None]


def _weights(pair, i, k, dtype):
    q, s = pair
    return _e4m3(q[i], s[i]) if s.dtype == FL else f4.decode(q[i], s[i], k, dtype)


def _choice(logits, top, renorm):
    """(experts, weights) in fp64; ties to the lower index, -inf never taken."""
    l = logits.double()
    val, ids = torch.sort(l, dim=1, descending=True, stable=True)
    val, ids = val[:, :top], ids[:, :top]
    none = val == float("-inf")
    peak = torch.where(none[:, :1], 0.0, val[:, :1])
    num = torch.where(none, 0.0, torch.exp(val - peak))
    den = num.sum(1, keepdim=True) if renorm else torch.exp(l - peak).sum(1, keepdim=True)
    return torch.where(none, -1, ids), torch.where(none, 0.0, num / torch.where(den > 0, den, 1.0))


def reference(x, logits, top, up, down, ub, db, renorm):
    """(out, bound)."""
    t, hidden = x.shape
    e = logits.shape[1]
    inner = up[0].shape[1] // 2
    h, tiny = f4.half_step(x.dtype), f4.tiny(x.dtype)
    ids, wts = _choice(logits, top, renorm)
    fin = logits.double()[torch.isfinite(logits)]
    spread = 2 * fin.abs().max().item() if fin.numel() else 0.0
    x64 = x.double()
    out = torch.zeros_like(x64)
    bound = torch.zeros_like(x64)
    total = torch.zeros_like(x64)
    for i in range(e):
        tok, place = (ids == i).nonzero(as_tuple=True)
        if not tok.numel():
            continue
        r, mag = f4.product(x64[tok], _weights(up, i, hidden, x.dtype), None if ub is None else ub[i])
        err = mag * (hidden + 8) * EPS
        g, u = r[:, :inner], r[:, inner:]
        eg, eu = err[:, :inner], err[:, inner:]
        silu = g * torch.sigmoid(g)
        act = silu * u
        ea = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + act.abs() * (h * (1 + 2.0 ** -8) + 12 * EPS) + tiny
        w = _weights(down, i, inner, x.dtype)
        y, mag = f4.product(act, w, None if db is None else db[i])
        ey = torch.mm(ea, w.abs().t().contiguous()) * (1 + inner * EPS) + mag * (inner + 8) * EPS
        wt = wts[tok, place, None]
        out.index_add_(0, tok, wt * y)
        total.index_add_(0, tok, wt * y.abs())
        bound.index_add_(0, tok, wt * ey + wt * y.abs() * (2 * spread + e + 16) * 2.0 ** -24)
    bound += total * (top + 24) * EPS + (out.abs() + bound) * h * (1 + 2.0 ** -8) + tiny
    return out, bound


def make(seed, fmt, t, e, top, hidden, inner, dtype, logits=FL, bias=False, masked=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    quantize = fw.quantize_fp4 if fmt == "fp4" else fw.quantize_experts
    up = quantize(rand(e, 2 * inner, hidden) / hidden ** 0.5)
    down = quantize(rand(e, hidden, inner) / inner ** 0.5)
    l = 2 * rand(t, e)
    if masked:
        l[torch.rand((t, e), generator=g, device=DEV) < masked] = float("-inf")
        l[3::7] = float("-inf")
    ub, db = (rand(e, 2 * inner).to(dtype), rand(e, hidden).to(dtype)) if bias else (None, None)
    return rand(t, hidden).to(dtype), l.to(logits), top, up, down, ub, db


def check(case, renorm=True, what=""):
    x, l, top, up, down, ub, db = case
    t, hidden = x.shape
    guard = torch.full((t + 2, hidden), float("nan"), dtype=x.dtype, device=DEV)
    need = fw.moe_layer_workspace_bytes(x, l, top, up)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)  # NaN wherever something unwritten is read
    fw.moe_layer(x, l, top, up, down, ub, db, renormalize=renorm, out=guard[1:-1], workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    assert (ws[need:] == 0xff).all(), "wrote outside the workspace"
    ref, bound = reference(x, l, top, up, down, ub, db, renorm)
    f4.assert_within(guard[1:-1], ref, bound, f"{what} t={t} e={l.shape[1]} top={top} hidden={hidden}")
    return guard[1:-1].clone()


CASES = [
    # fmt, t, e, top, hidden, inner, dtype, logits, bias, masked
    ("e4m3", 1, 8, 2, 512, 256, BF, BF, False, 0.0),
    ("fp4", 1, 8, 2, 512, 256, BF, FL, False, 0.0),
    ("e4m3", 1, 1, 1, 1, 1, HF, FL, True, 0.0),
    ("fp4", 1, 1, 1, 1, 1, BF, HF, True, 0.0),
    ("e4m3", 1, 128, 8, 1024, 384, BF, FL, False, 0.0),
    ("fp4", 1, 128, 8, 1024, 384, HF, BF, True, 0.0),
    ("e4m3", 3, 5, 5, 200, 77, HF, HF, True, 0.3),
    ("fp4", 3, 5, 5, 200, 77, HF, FL, True, 0.3),
    ("e4m3", 13, 60, 4, 1030, 513, HF, HF, True, 0.1),
    ("fp4", 13, 60, 4, 1030, 513, BF, HF, True, 0.1),
    ("e4m3", 16, 128, 8, 640, 320, BF, BF, False, 0.0),
    ("fp4", 16, 128, 8, 640, 320, BF, BF, False, 0.0),
    ("e4m3", 16, 2, 1, 333, 129, BF, FL, True, 0.0),
    ("fp4", 17, 2, 1, 333, 129, BF, FL, True, 0.0),
    ("e4m3", 20, 1, 1, 96, 1000, HF, FL, False, 0.0),
    ("fp4", 33, 1, 1, 96, 1000, HF, FL, False, 0.0),
    ("e4m3", 40, 3, 2, 260, 300, BF, HF, True, 0.2),
    ("fp4", 48, 3, 2, 260, 300, HF, HF, True, 0.2),
    ("e4m3", 64, 1, 1, 512, 512, BF, FL, True, 0.0),
    ("fp4", 64, 1, 1, 512, 512, BF, FL, True, 0.0),
    ("e4m3", 64, 8, 2, 1024, 896, BF, BF, False, 0.0),
    ("fp4", 64, 8, 2, 1024, 896, BF, BF, False, 0.0),
    ("e4m3", 64, 300, 8, 128, 64, BF, FL, False, 0.0),
    ("fp4", 64, 64, 64, 100, 40, HF, FL, True, 0.0),
    ("e4m3", 9, 1024, 3, 64, 32, BF, FL, True, 0.5),
    ("fp4", 30, 513, 6, 96, 33, BF, BF, False, 0.9),
    ("e4m3", 2, 4, 2, 64, 8200, BF, FL, False, 0.0),
    ("fp4", 2, 4, 2, 8200, 64, BF, FL, False, 0.0),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("fmt,t,e,top,hidden,inner,dtype,logits,bias,masked", CASES)
def test_layer(fmt, t, e, top, hidden, inner, dtype, logits, bias, masked, renorm):
    check(make(t + e + hidden, fmt, t, e, top, hidden, inner, dtype, logits, bias, masked), renorm, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64])
def test_layer_every_number_of_row_tiles(t, fmt):
    """All tokens to one expert, and half of them to another."""
    x, l, top, up, down, ub, db = make(t, fmt, t, 4, 2, 160, 96, BF, bias=True)
    l.zero_()
    l[:, 2] = 3.0
    l[::2, 0] = 2.0
    l[1::2, 0] = float("-inf")
    l[1::2, 1] = float("-inf")
    l[1::2, 3] = float("-inf")
    check((x, l, top, up, down, ub, db))


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_layer_padding_tokens_are_zeros(fmt):
    x, l, top, up, down, ub, db = make(5, fmt, 20, 8, 3, 128, 64, BF, bias=True)
    x[4], x[9] = float("nan"), float("inf")  # what stands in a padding token's row does not matter
    l[4] = l[9] = l[19] = float("-inf")
    out = fw.moe_layer(x, l, top, up, down, ub, db)
    assert (out[[4, 9, 19]] == 0).all() and torch.isfinite(out).all()
    l[:] = float("-inf")
    assert (fw.moe_layer(x, l, top, up, down, ub, db) == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_layer_nan_and_infinity_stay_in_their_tokens(fmt):
    x, l, top, up, down, ub, db = make(6, fmt, 20, 8, 2, 128, 64, BF)
    want = fw.moe_layer(x, l, top, up, down)
    x[3, 7], x[11, 100] = float("nan"), float("inf")
    l[15, 2] = float("nan")
    bad = torch.zeros(20, dtype=torch.bool, device=DEV)
    bad[[3, 11, 15]] = True
    out = fw.moe_layer(x, l, top, up, down)
    assert not torch.isfinite(out[bad]).all(dim=1).any() and torch.isnan(out[15]).all()
    assert torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_layer_is_its_parts(fmt):
    """route, the experts' products, the activation and the weighted sum: both within the bound of the same values, the
    parts' with their two further roundings per slot."""
    x, l, top, up, down, ub, db = make(7, fmt, 24, 8, 2, 256, 192, BF, BF, bias=True)
    product = fw.linear_experts_fp4 if fmt == "fp4" else fw.linear_experts
    r = fw.route(l, top)
    h = product(x, *up, r.offsets, ub, x_rows=r.tokens)
    act = (torch.nn.functional.silu(h[:, :192].float()) * h[:, 192:].float()).to(BF)
    parts = fw.combine(product(act, *down, r.offsets, db, y_rows=r.slots), r.weights)
    ref, bound = reference(x, l, top, up, down, ub, db, True)
    f4.assert_within(fw.moe_layer(x, l, top, up, down, ub, db), ref, bound, "layer")
    assert ((parts.double() - ref).norm() / ref.norm()).item() < 4 * f4.half_step(BF)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_layer_unaligned_buffers(fmt, off):
    x, l, top, up, down, ub, db = make(off, fmt, 6, 4, 2, 256, 256, HF, bias=True)

    def moved(t, by):
        by = (by + t.element_size() - 1) // t.element_size()
        buf = torch.full((t.numel() + 64,), 0x55, dtype=t.dtype, device=DEV)
        buf[by:by + t.numel()] = t.reshape(-1)
        return buf[by:by + t.numel()].view(t.shape)
    check((moved(x, off), moved(l, off), top, (moved(up[0], off), moved(up[1], off)),
           (moved(down[0], off), moved(down[1], off)), moved(ub, off), moved(db, off)))


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t", [1, 16, 40])
def test_layer_gives_the_same_bits_again(t, fmt):
    case = make(t, fmt, t, 32, 4, 512, 256, BF)
    want = fw.moe_layer(*case)
    for _ in range(10):
        assert torch.equal(fw.moe_layer(*case), want)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t", [1, 16, 40])
def test_layer_in_a_graph(t, fmt):
    """Replayed on other tokens, with eager calls between, against the eager results; two graphs share a workspace."""
    x, l, top, up, down, ub, db = make(t, fmt, t, 16, 2, 256, 320, BF, bias=True)
    ws = torch.empty(fw.moe_layer_workspace_bytes(x, l, top, up), dtype=torch.uint8, device=DEV)
    outs, graphs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fw.moe_layer(x, l, top, up, down, ub, db, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fw.moe_layer(x, l, top, up, down, ub, db, out=out, workspace=ws)
        outs.append(out)
        graphs.append(graph)
    for i in range(6):
        g = torch.Generator(device=DEV).manual_seed(100 + i)
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        l.copy_(torch.randn(l.shape, generator=g, device=DEV))
        want = fw.moe_layer(x, l, top, up, down, ub, db)
        for out, graph in zip(outs, graphs):
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_layer_on_other_streams(fmt):
    case = make(1, fmt, 12, 16, 2, 256, 320, BF)
    want = fw.moe_layer(*case)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(fw.moe_layer(*case))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_layer_no_tokens_and_too_many():
    x, l, top, up, down, ub, db = make(1, "fp4", 4, 4, 2, 64, 32, BF)
    assert fw.moe_layer(x[:0], l[:0], top, up, down).shape == (0, 64)
    many = torch.zeros((65, 64), dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="64 tokens"):
        fw.moe_layer(many, torch.zeros((65, 4), device=DEV), top, up, down)
