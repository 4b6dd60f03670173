"""Timed cases of the 4-bit operators and of the whole mixture-of-experts layer.

Three operators, as a serving program calls them:

  linear   the linear layer on 4-bit weights: e2m1 codes, two to a byte, with one
           power-of-two scale (e8m0) for 32 weights of a row; bf16 / fp16 activations
  experts  matrix products grouped by expert, ragged sizes, on such weights; the
           rows are gathered ("up") or scattered ("down") by the router's lists
  layer    a mixture-of-experts layer for a few tokens, from router logits and
           hidden states to the weighted sum of the experts' outputs: choice, gate
           and up products, silu(gate) * up, down products, weighted sum; weights
           in 4 bits, or e4m3 with a scale for each output channel

``own`` chooses between the plain form (elementary torch operations in 32 bits,
rounded once at the end) and this repository's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: one decoding token through a small layer, latency alone
        dict(name="linear_small", op="linear", m=1, n=1024, k=1024, dtype="fp16", bias=True),
        # one decoding token through a gate or up projection: the weights stream once
        dict(name="linear_token", op="linear", m=1, n=14336, k=4096, dtype="bf16", bias=False),
        # a decode batch through the down projection with its long rows
        dict(name="linear_batch", op="linear", m=22, n=4096, k=14336, dtype="bf16", bias=False),
        # a prompt through the gate or up projection: bound by the matrix cores
        dict(name="linear_prompt", op="linear", m=4096, n=14336, k=4096, dtype="bf16", bias=True),
        # down projection of a decode batch on many small experts: a few rows each, nearly all weights read
        dict(name="experts_batch", op="experts", side="down", t=64, e=128, top=8, n=4096, k=1024, dtype="bf16",
             bias=False, skew=1.0, masked=0.0),
        # odd sizes: rows of 500 1/2 bytes, a last scale for nine weights, empty experts, padding tokens, biases
        dict(name="experts_odd", op="experts", side="up", t=333, e=60, top=4, n=1030, k=1001, dtype="fp16",
             bias=True, skew=2.0, masked=0.05),
        # gate/up projection over a prompt, ragged groups
        dict(name="experts_prompt", op="experts", side="up", t=4096, e=8, top=2, n=14336, k=4096, dtype="bf16",
             bias=False, skew=0.5, masked=0.0),
        # one decoding token, two of eight large e4m3 experts
        dict(name="layer_token", op="layer", fmt="e4m3", t=1, e=8, top=2, hidden=4096, inner=14336, dtype="bf16",
             logits="bf16", bias=False, renorm=True, masked=0.0),
        # one decoding token, eight of many small 4-bit experts: little to read, so latency counts
        dict(name="layer_token_small", op="layer", fmt="fp4", t=1, e=128, top=8, hidden=4096, inner=1024, dtype="bf16",
             logits="fp32", bias=False, renorm=True, masked=0.0),
        # a decode batch over many small 4-bit experts: most of them have a row or two
        dict(name="layer_batch", op="layer", fmt="fp4", t=16, e=128, top=8, hidden=4096, inner=1024, dtype="bf16",
             logits="fp32", bias=False, renorm=True, masked=0.0),
        # odd widths, biases, padding tokens and forbidden experts
        dict(name="layer_odd", op="layer", fmt="e4m3", t=13, e=60, top=4, hidden=1030, inner=513, dtype="fp16",
             logits="fp16", bias=True, renorm=False, masked=0.1),
        # the largest decode batch that counts as a few tokens, on large e4m3 experts
        dict(name="layer_full", op="layer", fmt="e4m3", t=64, e=8, top=2, hidden=4096, inner=14336, dtype="bf16",
             logits="bf16", bias=False, renorm=True, masked=0.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer width: mostly multiples of 256 or 64, one in four whatever comes."""
    v = _log(rng, lo, hi)
    q = rng.choice([256, 256, 64, 1])
    return max(lo, v // q * q) if v >= q else v


def draw(rng):
    op = rng.choice(["linear", "linear", "experts", "layer", "layer"])
    if op == "linear":
        while True:
            c = dict(op=op, m=_log(rng, 1, 4096), n=_width(rng, 256, 14336), k=_width(rng, 256, 14336),
                     dtype=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5)
            if c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096:
                return c
    if op == "experts":
        while True:
            c = dict(op=op, side=rng.choice(["up", "down"]), t=_log(rng, 1, 4096), e=_log(rng, 2, 128),
                     top=rng.choice([1, 2, 4, 8]), n=_width(rng, 256, 14336), k=_width(rng, 256, 14336),
                     dtype=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5, skew=rng.choice([0.0, 1.0, 2.0]),
                     masked=rng.choice([0.0, 0.05]))
            if (c["top"] <= c["e"] and c["e"] * c["n"] * c["k"] <= 128 * 4096 * 1024
                    and c["t"] * c["top"] * c["n"] * c["k"] <= 8192 * 14336 * 4096):
                return c
    while True:
        c = dict(op=op, fmt=rng.choice(["fp4", "e4m3"]), t=_log(rng, 1, 64), e=_log(rng, 2, 128),
                 top=rng.choice([1, 2, 4, 8]), hidden=_width(rng, 1024, 8192), inner=_width(rng, 256, 14336),
                 dtype=rng.choice(["bf16", "fp16"]), logits=rng.choice(["bf16", "fp16", "fp32"]),
                 bias=rng.random() < 0.5, renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]))
        if c["top"] <= c["e"] and c["e"] * c["hidden"] * c["inner"] <= 128 * 4096 * 1024:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed))


def _activations(g, m, k, dtype):
    """N(0, 1) with one value in a thousand twenty times as large."""
    x = torch.randn((m, k), generator=g, device=g.device)
    x = torch.where(torch.rand((m, k), generator=g, device=g.device) < 1e-3, x * 20.0, x)
    return x.to(dtype)


def _fp4(w):
    """(codes, scales) of a weight [n, k]: e2m1 codes, the even k in the low four bits, and e8m0 scales 2^(s - 127),
    the largest power of two that the block's largest value holds four of (blocks of 32 along k, the last as it comes)."""
    n, k = w.shape
    blocks = torch.nn.functional.pad(w, (0, -k % 32)).view(n, -1, 32)
    ex = torch.frexp(blocks.abs().amax(dim=2)).exponent - 3  # amax = m 2^x with 1/2 <= m < 1
    v = torch.ldexp(blocks, -ex[:, :, None])
    mag = torch.bucketize(v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device))
    code = (mag + 8 * (v < 0)).to(torch.uint8).view(n, -1)[:, :k + k % 2]
    return code[:, 0::2] | (code[:, 1::2] << 4), (ex + 127).clamp(0, 254).to(torch.uint8)


def _stack(g, fmt, e, n, k):
    """e experts' weights [n, k], N(0, 0.02^2)."""
    if fmt == "fp4":
        q = torch.empty((e, n, (k + 1) // 2), dtype=torch.uint8, device="cuda")
        scale = torch.empty((e, n, (k + 31) // 32), dtype=torch.uint8, device="cuda")
    else:
        q = torch.empty((e, n, k), dtype=torch.uint8, device="cuda")
        scale = torch.empty((e, n), device="cuda")
    for i in range(e):
        w = 0.02 * torch.randn((n, k), generator=g, device="cuda")
        if fmt == "fp4":
            q[i], scale[i] = _fp4(w)
        else:
            amax = w.abs().amax(dim=1, keepdim=True)
            scale[i] = amax[:, 0] / 448.0
            q[i] = (w * (448.0 / amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return q, scale


def _choices(g, case):
    """Each token's distinct experts [t, top], -1 for padding tokens. ``skew`` tilts the load to the first experts."""
    t, e, top = case["t"], case["e"], case["top"]
    score = torch.randn((t, e), generator=g, device=g.device)
    score = score - case["skew"] * torch.arange(e, device=g.device) * (2.0 / e)
    ids = torch.topk(score, top, dim=1).indices
    pad = torch.rand((t, 1), generator=g, device=g.device) < case["masked"]
    return torch.where(pad, -1, ids)


def _lists(ids, e):
    """The slots (token * top + j) ordered by expert, padding slots last, and the experts' offsets."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, e, flat)
    slots = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(e, device=key.device)).sum(0)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=key.device)
    offsets[1:] = counts.cumsum(0).int()
    return slots.int(), offsets


def _logits(g, case):
    """Router logits; ``masked`` of them, and all of a padding token's (never the first), are -inf."""
    l = 2.0 * torch.randn((case["t"], case["e"]), generator=g, device=g.device)
    if case["masked"] > 0.0:
        hide = torch.rand(l.shape, generator=g, device=g.device) < case["masked"]
        hide[1:] |= torch.rand((case["t"] - 1, 1), generator=g, device=g.device) < 0.5 * case["masked"]
        l = l.masked_fill(hide, float("-inf"))
    return l.to(_DT[case["logits"]])


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], _DT[case["dtype"]]

    def bias(*shape):
        return (0.01 * torch.randn(shape, generator=g, device="cuda")).to(dt) if case["bias"] else None

    if op == "linear":
        q, scale = _stack(g, "fp4", 1, case["n"], case["k"])
        return dict(case=case, x=_activations(g, case["m"], case["k"], dt), q=q[0], scale=scale[0],
                    bias=bias(case["n"]))
    if op == "layer":
        e, h, i = case["e"], case["hidden"], case["inner"]
        return dict(case=case, x=_activations(g, case["t"], h, dt), logits=_logits(g, case),
                    gate_up=_stack(g, case["fmt"], e, 2 * i, h), down=_stack(g, case["fmt"], e, h, i),
                    gate_up_bias=bias(e, 2 * i), down_bias=bias(e, h))
    e, top, t = case["e"], case["top"], case["t"]
    q, scale = _stack(g, "fp4", e, case["n"], case["k"])
    slots, offsets = _lists(_choices(g, case), e)
    up = case["side"] == "up"
    return dict(case=case, x=_activations(g, t if up else t * top, case["k"], dt), q=q, scale=scale,
                bias=bias(e, case["n"]), offsets=offsets, ends=offsets.tolist(),
                x_rows=(slots // top).int() if up else None, y_rows=None if up else slots)


# ------------------------------------------------------------------ the plain form
def _weights(q, scale, k):
    """The weights [n, k] of codes and scales, in 32 bits (every value of both formats is exact)."""
    if scale.dtype == torch.float32:
        return q.view(torch.float8_e4m3fn).float() * scale[:, None]
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=q.device)
    n = q.shape[0]
    codes = torch.stack([q & 15, q >> 4], dim=2).view(n, -1)[:, :k]
    by = torch.exp2(scale.float() - 127.0).repeat_interleave(32, dim=1)[:, :k]
    return value[codes.int()] * by


def _plain_linear(s):
    y = s["x"].float() @ _weights(s["q"], s["scale"], s["case"]["k"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def _plain_experts(s):
    c, x = s["case"], s["x"]
    m = c["t"] * c["top"]
    xs = x.float() if s["x_rows"] is None else x[s["x_rows"].long()].float()
    y = torch.zeros((m, c["n"]), device=x.device)
    for i in range(c["e"]):
        lo, hi = s["ends"][i], s["ends"][i + 1]
        if hi > lo:
            r = xs[lo:hi] @ _weights(s["q"][i], s["scale"][i], c["k"]).t()
            y[lo:hi] = r if s["bias"] is None else r + s["bias"][i].float()
    y = y.to(x.dtype)
    if s["y_rows"] is None:
        return y
    out = torch.empty_like(y)
    out[s["y_rows"].long()] = y
    return out


def _choose(l, top, renorm):
    """Each token's experts by falling logit (-1: none left) and their weights, logits in 32 bits."""
    e = l.shape[1]
    idx = torch.arange(e, device=l.device)
    left, ids, vals = l.clone(), [], []
    for _ in range(top):
        best = left.amax(dim=1, keepdim=True)
        first = torch.where(left == best, idx, e).amin(dim=1, keepdim=True)
        ids.append(torch.where(best == float("-inf"), -1, first))
        vals.append(best)
        left = left.scatter(1, first, float("-inf"))
    ids, vals = torch.cat(ids, 1), torch.cat(vals, 1)
    peak = torch.where(vals[:, :1] == float("-inf"), 0.0, vals[:, :1])
    num = torch.exp(vals - peak)
    den = num.sum(1, keepdim=True) if renorm else torch.exp(l - peak).sum(1, keepdim=True)
    return ids, torch.where(ids < 0, 0.0, num / den)


def _plain_layer(s):
    c, x = s["case"], s["x"].float()
    i, h = c["inner"], c["hidden"]
    ids, weights = _choose(s["logits"].float(), c["top"], c["renorm"])
    out = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        if e < 0:
            continue
        tok, place = (ids == e).nonzero(as_tuple=True)
        r = x[tok] @ _weights(s["gate_up"][0][e], s["gate_up"][1][e], h).t()
        if c["bias"]:
            r = r + s["gate_up_bias"][e].float()
        a = r[:, :i] / (1.0 + torch.exp(-r[:, :i])) * r[:, i:]
        y = a @ _weights(s["down"][0][e], s["down"][1][e], i).t()
        if c["bias"]:
            y = y + s["down_bias"][e].float()
        out[tok] += weights[tok, place, None] * y  # a token is in an expert's list once
    return out.to(s["x"].dtype)


# ------------------------------------------------------------------ a pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "experts": _plain_experts, "layer": _plain_layer}[op](state)
    import fp8_weight_only_amd as fw
    if op == "linear":
        return fw.linear_fp4(state["x"], state["q"], state["scale"], state["bias"])
    if op == "experts":
        return fw.linear_experts_fp4(state["x"], state["q"], state["scale"], state["offsets"], state["bias"],
                                     x_rows=state["x_rows"], y_rows=state["y_rows"])
    return fw.moe_layer(state["x"], state["logits"], state["case"]["top"], state["gate_up"], state["down"],
                        state["gate_up_bias"], state["down_bias"], renormalize=state["case"]["renorm"])


# ------------------------------------------------------------------ the work of a pass
def _active(ids):
    """How many experts have rows."""
    return int(torch.unique(ids[ids >= 0]).numel())


def _weight_bytes(fmt, n, k):
    return n * ((k + 1) // 2 + (k + 31) // 32) if fmt == "fp4" else n * k + 4 * n


def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _weight_bytes("fp4", n, k) + 2 * (m * k + m * n + (n if case["bias"] else 0)),
                "flops": 2 * m * n * k}
    t, top = case["t"], case["top"]
    if op == "experts":
        n, k, m = case["n"], case["k"], t * top
        act = _active(_choices(_gen(1, "cpu"), case))
        rows_in = t if case["side"] == "up" else m
        return {"bytes": act * (_weight_bytes("fp4", n, k) + (2 * n if case["bias"] else 0))
                + 2 * (rows_in * k + m * n) + 4 * m, "flops": 2 * m * n * k}
    h, i = case["hidden"], case["inner"]
    l = _logits(_gen(1, "cpu"), case).float()
    best = torch.topk(l, top, dim=1)
    ids = torch.where(torch.isinf(best.values), -1, best.indices)
    rows = int((ids >= 0).sum())
    per = (_weight_bytes(case["fmt"], 2 * i, h) + _weight_bytes(case["fmt"], h, i)
           + (2 * (2 * i + h) if case["bias"] else 0))
    return {"bytes": max(1, _active(ids)) * per + 4 * t * h + t * case["e"] * (4 if case["logits"] == "fp32" else 2),
            "flops": max(1, rows) * 6 * h * i}


# ------------------------------------------------------------------ the definition in 64 bits
def _decode64(q, scale, k):
    """Weights [n, k] from the bits: sign, exponent and mantissa of each code."""
    if scale.dtype == torch.float32:
        c = q.long()
        ex, man = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * torch.pow(2.0, (ex - 10).double()))
        return torch.where(c >= 128, -mag, mag) * scale.double()[:, None]
    j = torch.arange(k, device=q.device)
    c = (q[:, j // 2].long() >> (4 * (j % 2))) & 15
    ex, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (2 + man) * torch.pow(2.0, (ex - 2).double()))
    return torch.where(c >= 8, -mag, mag) * torch.pow(2.0, scale[:, j // 32].double() - 127)


def _mm64(x, q, scale, k, bias):
    y = torch.mm(x, _decode64(q, scale, k).t().contiguous())
    return y if bias is None else y + bias.double()


def _exact_experts(s):
    c, x = s["case"], s["x"].double()
    m = c["t"] * c["top"]
    out = torch.zeros((m, c["n"]), dtype=torch.float64, device=x.device)
    place = torch.arange(m, device=x.device)
    src = place if s["x_rows"] is None else s["x_rows"].long()
    dst = place if s["y_rows"] is None else s["y_rows"].long()
    for i in range(c["e"]):
        rows = torch.arange(s["ends"][i], s["ends"][i + 1], device=x.device)
        if rows.numel():
            out[dst[rows]] = _mm64(x[src[rows]], s["q"][i], s["scale"][i], c["k"],
                                   None if s["bias"] is None else s["bias"][i])
    return out


def _exact_layer(s):
    c, x, l = s["case"], s["x"].double(), s["logits"].double()
    order = torch.sort(l, dim=1, descending=True, stable=True)
    ids, vals = order.indices[:, :c["top"]], order.values[:, :c["top"]]
    none = torch.isinf(vals)
    p = torch.exp(l - torch.where(none[:, :1], torch.zeros_like(vals[:, :1]), vals[:, :1]))
    share = torch.gather(p, 1, ids).masked_fill(none, 0.0)
    share = share / (share if c["renorm"] else p).sum(1, keepdim=True).clamp_min(1e-300)
    out = torch.zeros_like(x)
    for e in range(c["e"]):
        for j in range(c["top"]):
            tok = ((ids[:, j] == e) & ~none[:, j]).nonzero()[:, 0]
            if not tok.numel():
                continue
            r = _mm64(x[tok], s["gate_up"][0][e], s["gate_up"][1][e], c["hidden"],
                      s["gate_up_bias"][e] if c["bias"] else None)
            gate, up = r.chunk(2, dim=1)
            a = gate * torch.sigmoid(gate) * up
            y = _mm64(a, s["down"][0][e], s["down"][1][e], c["inner"], s["down_bias"][e] if c["bias"] else None)
            out.index_add_(0, tok, share[tok, j, None] * y)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _mm64(s["x"].double(), s["q"], s["scale"], case["k"], s["bias"])
    return _exact_experts(s) if case["op"] == "experts" else _exact_layer(s)
