"""Timed cases of the mixture-of-experts and int8 operators.

Four operators, as a serving program calls them:

  route    router logits -> each token's top experts, their weights, and the
           token slots ordered by expert (the row lists of the experts' products)
  experts  matrix products grouped by expert, ragged sizes, e4m3 weights with one
           scale per output channel, bf16 / fp16 activations; the rows are
           gathered ("up") or scattered ("down") by those lists
  combine  a token's weighted sum over its experts' outputs
  int8     the linear layer on 8-bit integers: weights with a scale for each
           output channel, activations quantized in the call with a scale for
           each token

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
        # one decoding token's router: latency alone
        dict(name="route_token", op="route", t=1, e=128, top=8, dtype="bf16", renorm=True, masked=0.0),
        # a decode batch on a small router, some experts masked out for some tokens
        dict(name="route_batch", op="route", t=250, e=8, top=2, dtype="fp16", renorm=False, masked=0.1),
        # the router over a long prompt with many experts
        dict(name="route_prompt", op="route", t=32768, e=256, top=8, dtype="fp32", renorm=True, masked=0.0),
        # gate/up projection of one decoding token: two experts' weights stream once
        dict(name="experts_token", op="experts", side="up", t=1, e=8, top=2, n=14336, k=4096, dtype="bf16",
             bias=False, skew=0.0, masked=0.0),
        # down projection of a decode batch on many small experts: a few rows each, nearly all weights read
        dict(name="experts_batch", op="experts", side="down", t=64, e=128, top=8, n=4096, k=1024, dtype="bf16",
             bias=False, skew=1.0, masked=0.0),
        # odd sizes: row lengths that no vector load divides, empty experts, padding tokens, biases
        dict(name="experts_odd", op="experts", side="up", t=333, e=60, top=4, n=1030, k=1001, dtype="fp16",
             bias=True, skew=2.0, masked=0.05),
        # gate/up projection over a prompt: bound by the matrix cores
        dict(name="experts_prompt", op="experts", side="up", t=4096, e=8, top=2, n=14336, k=4096, dtype="bf16",
             bias=False, skew=0.5, masked=0.0),
        # the weighted sum of a small decode batch
        dict(name="combine_batch", op="combine", t=22, top=2, n=4096, dtype="bf16"),
        # the weighted sum over a prompt
        dict(name="combine_prompt", op="combine", t=8192, top=8, n=4096, dtype="bf16"),
        # one decoding token through an int8 layer
        dict(name="int8_token", op="int8", m=1, n=14336, k=4096, dtype="bf16", bias=True),
        # a decode batch through the narrow layer with the long rows
        dict(name="int8_batch", op="int8", m=22, n=4096, k=14336, dtype="fp16", bias=False),
        # a prompt through an int8 layer: bound by the matrix cores
        dict(name="int8_prompt", op="int8", m=4096, n=14336, k=4096, dtype="bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer width: mostly multiples of 256 or 64, one in four whatever comes."""
    v = _log(rng, lo, hi)
    q = rng.choice([256, 256, 64, 1])
    return max(lo, v // q * q) if v >= q else v


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "combine", "int8", "int8"])
    if op == "route":
        e = _log(rng, 4, 256)
        return dict(op=op, t=_log(rng, 1, 32768), e=e, top=rng.randint(1, min(8, e)),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), renorm=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.1, 0.5]))
    if op == "experts":
        while True:
            c = dict(op=op, side=rng.choice(["up", "down"]), t=_log(rng, 1, 4096), e=_log(rng, 2, 128),
                     top=rng.choice([1, 2, 4, 8]), n=_width(rng, 256, 14336), k=_width(rng, 256, 14336),
                     dtype=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5, skew=rng.choice([0.0, 1.0, 2.0]),
                     masked=rng.choice([0.0, 0.05]))
            if (c["top"] <= c["e"] and c["e"] * c["n"] * c["k"] <= 128 * 4096 * 1024
                    and c["t"] * c["top"] * c["n"] * c["k"] <= 8192 * 14336 * 4096):
                return c
    if op == "combine":
        while True:
            c = dict(op=op, t=_log(rng, 1, 8192), top=rng.choice([1, 2, 3, 4, 6, 8]), n=_width(rng, 256, 8192),
                     dtype=rng.choice(["bf16", "fp16"]))
            if c["t"] * c["top"] * c["n"] <= 8192 * 8 * 4096:
                return c
    while True:
        c = dict(op=op, m=_log(rng, 1, 4096), n=_width(rng, 256, 14336), k=_width(rng, 256, 14336),
                 dtype=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5)
        if c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed))


def _activations(g, m, k, dtype):
    """N(0, 1) with one value in a thousand twenty times as large."""
    x = torch.randn((m, k), generator=g, device=g.device)
    x = torch.where(torch.rand((m, k), generator=g, device=g.device) < 1e-3, x * 20.0, x)
    return x.to(dtype)


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


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "route":
        logits = 2.0 * torch.randn((case["t"], case["e"]), generator=g, device="cuda")
        if case["masked"] > 0.0:  # experts a token may not take; now and then all of them (padding)
            hide = torch.rand(logits.shape, generator=g, device="cuda") < case["masked"]
            hide |= torch.rand((case["t"], 1), generator=g, device="cuda") < 0.02
            logits = logits.masked_fill(hide, float("-inf"))
        return dict(case=case, logits=logits.to(dt))
    if op == "combine":
        y = torch.randn((case["t"] * case["top"], case["n"]), generator=g, device="cuda").to(dt)
        w = torch.softmax(torch.randn((case["t"], case["top"]), generator=g, device="cuda"), dim=1)
        return dict(case=case, y=y, w=w)
    n, k = case["n"], case["k"]
    bias = (0.01 * torch.randn((n,), generator=g, device="cuda")).to(dt) if op == "int8" and case["bias"] else None
    if op == "int8":
        w = 0.02 * torch.randn((n, k), generator=g, device="cuda")
        amax = w.abs().amax(dim=1, keepdim=True)
        q = torch.round(w * (127.0 / amax)).clamp(-127, 127).to(torch.int8)
        return dict(case=case, x=_activations(g, case["m"], k, dt), q=q, scale=(amax / 127.0)[:, 0], bias=bias)
    e, top, t = case["e"], case["top"], case["t"]
    q = torch.empty((e, n, k), dtype=torch.uint8, device="cuda")
    scale = torch.empty((e, n), device="cuda")
    for i in range(e):
        w = 0.02 * torch.randn((n, k), generator=g, device="cuda")
        amax = w.abs().amax(dim=1, keepdim=True)
        scale[i] = amax[:, 0] / 448.0
        q[i] = (w * (448.0 / amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    if case["bias"]:
        bias = (0.01 * torch.randn((e, n), generator=g, device="cuda")).to(dt)
    slots, offsets = _lists(_choices(g, case), e)
    up = case["side"] == "up"
    return dict(case=case, x=_activations(g, t if up else t * top, k, dt), q=q, scale=scale, bias=bias,
                offsets=offsets, ends=offsets.tolist(),
                x_rows=(slots // top).int() if up else None, y_rows=None if up else slots)


# ------------------------------------------------------------------ the plain form
def _plain_route(s):
    c, l = s["case"], s["logits"].float()
    t, e, top = c["t"], c["e"], c["top"]
    idx = torch.arange(e, device=l.device)
    left, ids, vals = l.clone(), [], []
    for _ in range(top):
        best = left.amax(dim=1, keepdim=True)
        first = torch.where(left == best, idx, e).amin(dim=1, keepdim=True)
        ids.append(torch.where(best == float("-inf"), -1, first))
        vals.append(best)
        left = left.scatter(1, first, float("-inf"))
    ids, vals = torch.cat(ids, 1), torch.cat(vals, 1)
    peak = vals[:, :1]
    safe = torch.where(peak == float("-inf"), 0.0, peak)
    num = torch.exp(vals - safe)
    den = num.sum(1, keepdim=True) if c["renorm"] else torch.exp(l - safe).sum(1, keepdim=True)
    weights = torch.where(ids < 0, 0.0, num / den)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, e, flat)
    slots = torch.sort(key, stable=True).indices
    counts = torch.zeros(e + 1, dtype=torch.int64, device=l.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=l.device)
    offsets[1:] = counts[:e].cumsum(0).int()
    return weights, ids.int(), offsets, slots.int(), (slots // top).int()


def _plain_experts(s):
    c, x = s["case"], s["x"]
    m = c["t"] * c["top"]
    xs = x.float() if s["x_rows"] is None else x[s["x_rows"].long()].float()
    y = torch.zeros((m, c["n"]), device=x.device)
    for i in range(c["e"]):
        lo, hi = s["ends"][i], s["ends"][i + 1]
        if hi > lo:
            w = s["q"][i].view(torch.float8_e4m3fn).float()
            r = (xs[lo:hi] @ w.t()) * s["scale"][i]
            y[lo:hi] = r if s["bias"] is None else r + s["bias"][i].float()
    y = y.to(x.dtype)
    if s["y_rows"] is None:
        return y
    out = torch.empty_like(y)
    out[s["y_rows"].long()] = y
    return out


def _plain_combine(s):
    c = s["case"]
    y = s["y"].float().view(c["t"], c["top"], c["n"])
    return (y * s["w"][:, :, None]).sum(1).to(s["y"].dtype)


def _plain_int8(s):
    x = s["x"].float()
    amax = x.abs().amax(dim=1, keepdim=True)
    codes = torch.where(amax > 0.0, torch.round(x * 127.0 / amax), 0.0)  # 127 x is exact, the quotient rounded once
    y = (codes @ s["q"].float().t()) * (amax / 127.0) * s["scale"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


# ------------------------------------------------------------------ a pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"route": _plain_route, "experts": _plain_experts, "combine": _plain_combine,
                "int8": _plain_int8}[op](state)
    import fp8_weight_only_amd as fw
    if op == "route":
        r = fw.route(state["logits"], state["case"]["top"], renormalize=state["case"]["renorm"])
        return r.weights, r.experts, r.offsets, r.slots, r.tokens
    if op == "experts":
        return fw.linear_experts(state["x"], state["q"], state["scale"], state["offsets"], state["bias"],
                                 x_rows=state["x_rows"], y_rows=state["y_rows"])
    if op == "combine":
        return fw.combine(state["y"], state["w"])
    return fw.linear_int8(state["x"], state["q"], state["scale"], state["bias"])


# ------------------------------------------------------------------ the work of a pass
def _active(case):
    """How many experts have rows, for a load drawn like the case's."""
    ids = _choices(_gen(1, "cpu"), case)
    return int(torch.unique(ids[ids >= 0]).numel())


def work(case):
    op = case["op"]
    eb = 4 if case["dtype"] == "fp32" else 2
    if op == "route":
        t, e, top = case["t"], case["e"], case["top"]
        return {"bytes": t * e * eb + 16 * t * top + 4 * (e + 1), "flops": 4 * t * e}
    if op == "combine":
        t, top, n = case["t"], case["top"], case["n"]
        return {"bytes": t * (top + 1) * n * eb + 4 * t * top, "flops": 2 * t * top * n}
    n, k = case["n"], case["k"]
    if op == "int8":
        m = case["m"]
        return {"bytes": n * k + 4 * n + (m * k + m * n + (n if case["bias"] else 0)) * eb, "flops": 2 * m * n * k}
    m, act = case["t"] * case["top"], _active(case)
    rows_in = case["t"] if case["side"] == "up" else m
    return {"bytes": act * (n * k + 4 * n + (n * eb if case["bias"] else 0)) + (rows_in * k + m * n) * eb + 4 * m,
            "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_route(s):
    c, l = s["case"], s["logits"].double()
    t, e, top = c["t"], c["e"], c["top"]
    order = torch.sort(l, dim=1, descending=True, stable=True)
    vals, ids = order.values[:, :top], order.indices[:, :top]
    off = torch.isinf(vals)
    p = torch.exp(l - torch.where(off[:, :1], torch.zeros_like(vals[:, :1]), vals[:, :1]))
    chosen = torch.gather(p, 1, ids).masked_fill(off, 0.0)
    total = chosen.sum(1) if c["renorm"] else p.sum(1)
    weights = (chosen / total.clamp_min(1e-300)[:, None])
    ids = ids.masked_fill(off, -1)
    slots, offsets = _lists(ids, e)
    return weights, ids.int(), offsets, slots, torch.div(slots, top, rounding_mode="floor").int()


def _exact_experts(s):
    c, x = s["case"], s["x"].double()
    m = c["t"] * c["top"]
    out = torch.zeros((m, c["n"]), dtype=torch.float64, device=x.device)
    place = torch.arange(m, device=x.device)
    src = place if s["x_rows"] is None else s["x_rows"].long()
    dst = place if s["y_rows"] is None else s["y_rows"].long()
    code = torch.arange(256, device=x.device)
    ex, man = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(ex == 0, man * 2.0 ** -9, (1 + man / 8) * torch.pow(2.0, (ex - 7).double()))
    value = torch.where(code >= 128, -mag, mag)
    offsets = s["offsets"].long()
    for i in range(c["e"]):
        rows = torch.arange(int(offsets[i]), int(offsets[i + 1]), device=x.device)
        if rows.numel() == 0:
            continue
        w = value[s["q"][i].long()] * s["scale"][i].double()[:, None]
        r = torch.mm(x[src[rows]], w.t().contiguous())
        if s["bias"] is not None:
            r += s["bias"][i].double()
        out[dst[rows]] = r
    return out


def _exact_int8(s):
    x = s["x"].double()
    amax = x.abs().max(dim=1).values
    ratio = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    near = x * ratio[:, None]
    # x * 127 / amax is a fraction with a short denominator: within 1e-9 of a half it is a half
    half = torch.floor(near) + 0.5
    near = torch.where((near - half).abs() < 1e-9, half, near)
    y = torch.mm(torch.round(near), s["q"].double().t().contiguous())
    y *= (amax / 127.0)[:, None] * s["scale"].double()[None, :]
    return y if s["bias"] is None else y + s["bias"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "experts":
        return _exact_experts(s)
    if case["op"] == "combine":
        y = s["y"].double().view(case["t"], case["top"], case["n"])
        out = torch.zeros((case["t"], case["n"]), dtype=torch.float64, device=y.device)
        for j in range(case["top"]):
            out += s["w"][:, j, None].double() * y[:, j]
        return out
    return _exact_int8(s)
