"""GPU parity of routing, products grouped by expert, their weighted sum and the
int8 layer against plain 64-bit computations.

Tolerances count roundings. An output rounded to a type with p significant bits
is off by 2^-p of its value at most (bf16 2^-8 before the leading bit's weight,
that is eps / 2; fp16 2^-11), an fp32 operation by 2^-24, a product chained
through the matrix cores by up to 2^-23 (they may truncate) of the magnitudes
summed.
"""
import numpy as np
import pytest
import torch

import fp8_weight_only_amd as fw
import oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _tiny(dtype):
    """Half the spacing of the smallest values of a type."""
    return {BF: 2.0 ** -134, HF: 2.0 ** -25}[dtype]


def _assert_within(y, ref, tol, what):
    y = np.asarray(y, dtype=np.float64)
    assert np.isfinite(y).all(), f"{what}: non-finite outputs"
    bad = np.argwhere(np.abs(y - ref) > tol)
    if len(bad):
        i = tuple(bad[0])
        raise AssertionError(f"{what}: {len(bad)} of {ref.size} outside; first at {i}: {y[i]!r} against {ref[i]!r}, "
                             f"tolerance {tol[i]!r}")


# ------------------------------------------------------------------ route
def _route_ref(logits, top, renorm):
    """Choice and lists by Python's stable sort, weights in fp64; finite logits and -inf."""
    l = logits.double().cpu().numpy()
    t, e = l.shape
    weights, experts = np.zeros((t, top)), np.full((t, top), -1)
    for i in range(t):
        order = sorted((j for j in range(e) if l[i, j] != -np.inf), key=lambda j: (-l[i, j], j))[:top]
        if not order:
            continue
        p = np.exp(l[i] - l[i, order[0]])
        experts[i, :len(order)] = order
        weights[i, :len(order)] = p[order] / (p[order].sum() if renorm else p.sum())
    flat = experts.reshape(-1)
    slots = np.array(sorted(range(t * top), key=lambda s: (flat[s] if flat[s] >= 0 else e, s)), dtype=np.int64)
    offsets = np.array([0, *np.cumsum([(flat == i).sum() for i in range(e)])])
    return weights, experts, offsets, slots


def _check_route(logits, top, renorm):
    e = logits.shape[1]
    r = fw.route(logits, top, renormalize=renorm)
    torch.cuda.synchronize()
    weights, experts, offsets, slots = _route_ref(logits, top, renorm)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.array_equal(r.tokens.cpu().numpy(), slots // top)
    # exp: its argument's rounding (|difference| 2^-24), the function's own two steps; the sum's e roundings; the quotient
    fin = logits.double().cpu().numpy()
    spread = np.where(np.isfinite(fin), fin, 0.0)
    d = 2 * np.abs(spread).max() if spread.size else 0.0
    tol = weights * (2 * d + e + 16) * 2.0 ** -24 + 1e-37
    _assert_within(r.weights.cpu().numpy(), weights, tol, "weights")
    return r


ROUTES = [(1, 128, 8, BF), (1, 1, 1, FL), (3, 2, 2, HF), (22, 8, 2, BF), (17, 60, 4, FL), (250, 65, 6, HF),
          (100, 129, 8, FL), (40, 300, 5, BF), (64, 1024, 64, FL), (1000, 256, 8, FL), (5001, 64, 3, BF),
          (33, 64, 64, HF), (700, 1024, 1, BF)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,top,dtype", ROUTES)
def test_route(t, e, top, dtype, renorm):
    g = torch.Generator().manual_seed(t + e)
    _check_route((2.0 * torch.randn((t, e), generator=g)).to(dtype).to(DEV), top, renorm)


@pytest.mark.parametrize("t,e,top", [(300, 16, 4), (9, 200, 3), (2000, 8, 8)])
def test_route_masked_experts_padding_tokens_and_ties(t, e, top):
    g = torch.Generator().manual_seed(t)
    logits = torch.randint(-3, 3, (t, e), generator=g).float()  # many ties
    logits[logits == 0] = torch.where(torch.rand(int((logits == 0).sum()), generator=g) < 0.5, 0.0, -0.0)
    logits[torch.rand((t, e), generator=g) < 0.6] = float("-inf")
    logits[::7] = float("-inf")
    r = _check_route(logits.to(DEV), top, True)
    assert (r.experts[::7] == -1).all() and (r.weights[::7] == 0).all()


def test_route_all_tokens_to_one_expert_and_none_at_all():
    logits = torch.zeros((3000, 40), device=DEV)
    logits[:, 17] = 1.0
    _check_route(logits, 1, True)
    _check_route(torch.full((200, 40), float("-inf"), device=DEV), 2, False)


def test_route_nan_and_infinity():
    logits = torch.zeros((4, 8), device=DEV)
    logits[0, 3] = float("nan")
    logits[1, 5] = float("inf")
    logits[2, :] = float("-inf")
    logits[2, 6] = -1e30
    r = fw.route(logits, 2)
    assert r.experts.cpu().tolist() == [[3, 0], [5, 0], [6, -1], [0, 1]]
    w = r.weights.cpu()
    assert torch.isnan(w[0]).all() and torch.isnan(w[1]).all()
    assert w[2].tolist() == [1.0, 0.0] and w[3].tolist() == [0.5, 0.5]


def test_route_no_tokens():
    r = fw.route(torch.zeros((0, 12), device=DEV), 3)
    assert r.offsets.cpu().tolist() == [0] * 13 and r.slots.numel() == 0


def test_route_extreme_spread():
    logits = torch.tensor([[0.0, -200.0, 3e38, -3e38], [88.0, -88.0, 0.0, 1e-40]], device=DEV)
    r = fw.route(logits, 4, renormalize=False)
    assert r.experts.cpu().tolist() == [[2, 0, 1, 3], [0, 3, 2, 1]]
    assert r.weights[0].cpu().tolist() == [1.0, 0.0, 0.0, 0.0]


# ------------------------------------------------------------------ experts
def _lengths(rng, m, e, kind):
    """Ragged group sizes with sum <= m."""
    if kind == "one":
        n = np.zeros(e, dtype=int)
        n[e // 2] = m
        return n
    p = rng.dirichlet(np.full(e, 0.3 if kind == "skew" else 5.0))
    n = rng.multinomial(m, p)
    if kind == "tail":
        n[-1] = 0
        n = n // 2
    return n


def _experts_case(seed, m, e, n, k, dtype, bias, kind, gather, scatter, xr=None):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((e * n, k)) * 0.02).astype(np.float32)
    q, s = fw.quantize(torch.from_numpy(w).to(DEV))
    xr = (xr or max(1, m // 2)) if gather else m
    x = torch.from_numpy(rng.standard_normal((xr, k)).astype(np.float32)).to(dtype).to(DEV)
    b = torch.from_numpy(rng.standard_normal((e, n)).astype(np.float32)).to(dtype).to(DEV) if bias else None
    lens = _lengths(rng, m, e, kind)
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    xi = rng.integers(0, xr, m).astype(np.int32) if gather else None
    yi = rng.permutation(m).astype(np.int32) if scatter else None
    return x, q.view(e, n, k), s.view(e, n), b, offsets, xi, yi


def _dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def _experts_ref(x, q, s, b, offsets, xi, yi, m):
    """(y, sum of magnitudes) in fp64."""
    e, n, k = q.shape
    x64 = x.double().cpu().numpy()
    y, mag = np.zeros((m, n)), np.zeros((m, n))
    s64 = s.double().cpu().numpy()
    for i in range(e):
        p = np.arange(offsets[i], offsets[i + 1])
        if len(p) == 0:
            continue
        w = oracle.decode(np.ascontiguousarray(q[i].cpu().numpy())).reshape(n, k)
        rows = x64[p if xi is None else xi[p]]
        dst = p if yi is None else yi[p]
        y[dst] = rows @ w.T * s64[i]
        mag[dst] = np.abs(rows) @ np.abs(w).T * s64[i]
        if b is not None:
            y[dst] += b[i].double().cpu().numpy()
            mag[dst] += np.abs(b[i].double().cpu().numpy())
    return y, mag


def _experts_tol(y, mag, k, dtype):
    return np.abs(y) * _half_step(dtype) * (1 + 2.0 ** -8) + mag * (k + 8) * 2.0 ** -23 + _tiny(dtype)


def _check_experts(case, m):
    x, q, s, b, offsets, xi, yi = case
    n, k = q.shape[1:]
    guard = torch.full((m + 2, n), float("nan"), dtype=x.dtype, device=DEV)
    y = fw.linear_experts(x, q, s, _dev(offsets), b, _dev(xi), _dev(yi), out=guard[1:-1])
    torch.cuda.synchronize()
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    ref, mag = _experts_ref(x, q, s, b, offsets, xi, yi, m)
    _assert_within(y.double().cpu().numpy(), ref, _experts_tol(ref, mag, k, x.dtype),
                   f"experts {tuple(q.shape)} m={m} {fw.fp8w_linear_experts_kernel(m, *q.shape, 0, 0)}")
    return y


EXPERTS = [
    # m, e, n, k, dtype, bias, kind, gather, scatter
    (1, 1, 1, 1, BF, True, "even", False, False),
    (2, 8, 512, 1024, BF, False, "even", True, False),
    (1, 4, 300, 4096, HF, True, "even", False, True),
    (8, 64, 128, 512, BF, False, "even", True, False),
    (5, 3, 40, 17, HF, True, "skew", True, True),
    (64, 16, 256, 256, HF, False, "even", True, False),
    (100, 60, 130, 77, BF, True, "skew", True, False),
    (130, 7, 1030, 1001, HF, True, "tail", False, True),
    (129, 2, 64, 64, BF, False, "one", False, False),
    (300, 8, 264, 512, HF, True, "skew", True, False),
    (512, 5, 512, 768, BF, False, "tail", True, True),
    (700, 3, 200, 320, BF, True, "skew", False, False),
    (333, 1, 257, 256, HF, False, "even", False, True),
    (40, 1024, 16, 64, BF, False, "even", True, False),
    (65, 130, 96, 128, HF, True, "skew", True, True),
    (1500, 4, 768, 256, BF, True, "even", True, False),
    (32, 2, 96, 8192, BF, False, "even", False, False),
    (48, 3, 80, 2048, HF, True, "even", True, True),
]


@pytest.mark.parametrize("m,e,n,k,dtype,bias,kind,gather,scatter", EXPERTS)
def test_linear_experts(m, e, n, k, dtype, bias, kind, gather, scatter):
    _check_experts(_experts_case(m + n, m, e, n, k, dtype, bias, kind, gather, scatter), m)


@pytest.mark.parametrize("m", [3, 90, 600])
@pytest.mark.parametrize("qoff,xoff", [(8, 0), (1, 0), (0, 8), (0, 2), (3, 6)])
def test_linear_experts_unaligned_buffers(m, qoff, xoff):
    x, q, s, b, offsets, xi, yi = _experts_case(m, m, 4, 96, 512, BF, True, "even", True, False)
    qb = torch.empty(q.numel() + 64, dtype=torch.uint8, device=DEV)
    qb[qoff:qoff + q.numel()] = q.reshape(-1)
    xb = torch.empty(x.numel() + 64, dtype=BF, device=DEV)
    xb[xoff // 2:xoff // 2 + x.numel()] = x.reshape(-1)
    q2 = qb[qoff:qoff + q.numel()].view(q.shape)
    x2 = xb[xoff // 2:xoff // 2 + x.numel()].view(x.shape)
    _check_experts((x2, q2, s, b, offsets, xi, yi), m)


@pytest.mark.parametrize("m,n,k", [(6, 64, 512), (200, 128, 256), (40, 33, 100)])
def test_linear_experts_bad_rows_and_offsets(m, n, k):
    """Device values out of range: rows of NaN, rows not written, offsets clamped; no byte outside the buffers."""
    x, q, s, b, offsets, xi, yi = _experts_case(m, m, 4, n, k, BF, False, "even", True, True)
    xi[1], xi[m - 1], yi_bad = 1 << 30, -1, yi.copy()
    lost = yi[2]
    yi_bad[2], yi_bad[0] = -5, m
    guard = torch.full((m + 2, n), 7.0, dtype=BF, device=DEV)
    fw.linear_experts(x, q, s, _dev(offsets), b, _dev(xi), _dev(yi_bad), out=guard[1:-1])
    y = guard[1:-1].float().cpu().numpy()
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    assert np.isnan(y[yi[1]]).all() and np.isnan(y[yi[m - 1]]).all()
    assert (y[lost] == 7).all() and (y[yi[0]] == 7).all()
    wild = np.array([-9, 1 << 30, 2, m + 50, -(1 << 31)], dtype=np.int32)
    guard.fill_(7.0)
    fw.linear_experts(x, q, s, _dev(wild), None, None if x.shape[0] == m else _dev(xi), None, out=guard[1:-1])
    torch.cuda.synchronize()
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()


def test_linear_experts_no_rows_no_width():
    x, q, s, b, offsets, _, _ = _experts_case(1, 4, 3, 16, 0, BF, True, "even", False, False)
    y = fw.linear_experts(x, q, s, _dev(offsets), b)
    for i in range(3):  # k == 0: the bias
        assert torch.equal(y[offsets[i]:offsets[i + 1]], b[i].expand(offsets[i + 1] - offsets[i], -1))
    assert fw.linear_experts(x[:0], q, s, torch.zeros(4, dtype=torch.int32, device=DEV)).shape == (0, 16)
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert (fw.linear_experts(x, q, s, none, b) == 0).all()  # every row without an expert


def test_linear_experts_nan_stays_in_its_rows():
    x, q, s, b, offsets, _, _ = _experts_case(3, 70, 3, 96, 256, BF, False, "even", False, False)
    x[11, 5] = float("nan")
    x[40, 9] = float("inf")
    y = fw.linear_experts(x, q, s, _dev(offsets)).float().cpu()
    bad = ~torch.isfinite(y).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [11, 40]


def test_linear_experts_against_the_linear_layer():
    """One expert is the FP8 linear layer: both within the tolerance of the same 64-bit values."""
    x, q, s, b, offsets, _, _ = _experts_case(5, 96, 1, 512, 1024, BF, True, "even", False, False)
    ref, mag = _experts_ref(x, q, s, b, offsets, None, None, 96)
    tol = _experts_tol(ref, mag, 1024, BF)
    for y in (fw.linear(x, q[0], s[0], b[0]), fw.linear_experts(x, q, s, _dev(offsets), b)):
        _assert_within(y.double().cpu().numpy(), ref, tol, "linear")


def test_linear_experts_short_workspace_still_runs():
    x, q, s, b, offsets, xi, _ = _experts_case(8, 2, 8, 128, 4096, BF, True, "even", True, False)
    ref, mag = _experts_ref(x, q, s, b, offsets, xi, None, 2)
    y = fw.linear_experts(x, q, s, _dev(offsets), b, _dev(xi), workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    _assert_within(y.double().cpu().numpy(), ref, _experts_tol(ref, mag, 4096, BF), "no workspace")


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("t,top,n,dtype", [(1, 1, 1, BF), (22, 2, 4096, BF), (7, 8, 1001, HF), (300, 3, 263, BF),
                                           (5, 64, 16, HF), (64, 4, 2056, HF), (2, 0, 40, BF), (129, 6, 8, BF)])
def test_combine(t, top, n, dtype):
    g = torch.Generator().manual_seed(t + n)
    y = torch.randn((t * top, n), generator=g).to(dtype)
    w = torch.randn((t, top), generator=g)
    out = torch.full((t + 2, n), float("nan"), dtype=dtype, device=DEV)
    fw.combine(y.to(DEV), w.to(DEV), out=out[1:-1])
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all()
    terms = y.double().view(t, top, n) * w.double()[:, :, None]
    ref = terms.sum(1).numpy()
    tol = np.abs(ref) * _half_step(dtype) * (1 + 2.0 ** -8) + terms.abs().sum(1).numpy() * (top + 1) * 2.0 ** -24
    _assert_within(out[1:-1].double().cpu().numpy(), ref, tol + _tiny(dtype), "combine")


def test_combine_infinity_and_nan():
    y = torch.zeros((4, 8), dtype=BF, device=DEV)
    y[1, 2], y[2, 3] = float("inf"), float("nan")
    out = fw.combine(y, torch.tensor([[1.0, 0.5], [0.5, 0.5]], device=DEV)).float().cpu()
    assert out[0, 2] == float("inf") and torch.isnan(out[1, 3]) and torch.isfinite(out).sum() == 14


# ------------------------------------------------------------------ int8
def _codes_ref(x64):
    """Nearest integers (ties to even) of 127 x / amax in exact arithmetic: a quotient that is no half is over 1e-9 away."""
    amax = np.abs(x64).max(axis=1, keepdims=True) if x64.shape[1] else np.zeros((x64.shape[0], 1))
    r = 127.0 * x64 / np.where(amax > 0, amax, 1.0)
    half = np.floor(r) + 0.5
    r = np.where(np.abs(r - half) < 1e-9, half, r)
    return np.rint(r), amax[:, 0]


@pytest.mark.parametrize("m,k,dtype", [(1, 4096, BF), (5, 1001, HF), (300, 256, BF), (33, 14336, HF), (2, 1, BF),
                                       (64, 64, HF), (3, 20000, BF)])
def test_quantize_activations_int8(m, k, dtype):
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn((m, k), generator=g) * 10.0 ** torch.randint(-4, 4, (m, 1), generator=g)
    x = x.to(dtype)
    if m > 1:
        x[1] = 0.0
    qx, sx = fw.quantize_activations_int8(x.to(DEV))
    codes, amax = _codes_ref(x.double().numpy())
    assert np.array_equal(qx.cpu().numpy(), codes)
    assert np.array_equal(sx.cpu().numpy(), amax.astype(np.float32) / np.float32(127.0))


def test_quantize_activations_int8_ties_and_extremes():
    """Every ratio j / 254 of the maximum (the odd ones are ties), at ordinary, huge and tiny magnitudes."""
    for dtype, mags in ((BF, [1.0, 2.0 ** 119, 2.0 ** -120, 2.0 ** -140]), (HF, [1.0, 2.0 ** 8, 2.0 ** -14])):
        for mag in mags:
            j = torch.arange(-254, 255, dtype=torch.float64)
            x = (j * mag).to(dtype)[None]
            qx, sx = fw.quantize_activations_int8(x.to(DEV))
            codes, amax = _codes_ref(x.double().numpy())
            assert np.array_equal(qx.cpu().numpy(), codes), (dtype, mag)
    top = torch.tensor([[3.3895e38, -3.3895e38, 1.0, 1.7e38]]).to(BF)
    qx, _ = fw.quantize_activations_int8(top.to(DEV))
    assert np.array_equal(qx.cpu().numpy(), _codes_ref(top.double().numpy())[0])


def _int8_case(seed, m, n, k, dtype, bias):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((n, k), generator=g) * 0.02
    q, s = fw.quantize_int8(w.to(DEV))
    x = torch.randn((m, k), generator=g)
    x[torch.rand((m, k), generator=g) < 1e-3] *= 20.0
    b = torch.randn((n,), generator=g).to(dtype) if bias else None
    return x.to(dtype), q, s, b


def _int8_ref(x, q, s, b):
    codes, amax = _codes_ref(x.double().numpy())
    prod = (codes @ q.cpu().numpy().astype(np.float64).T) * (amax / 127.0)[:, None] * s.double().cpu().numpy()[None, :]
    y = prod if b is None else prod + b.double().numpy()[None, :]
    # the sum to fp32, the token scale, its product, the fused multiply-add's: within five fp32 roundings
    dt = x.dtype
    return y, np.abs(y) * _half_step(dt) * (1 + 2.0 ** -8) + np.abs(prod) * 5 * 2.0 ** -24 + _tiny(dt)


INT8 = [(1, 1024, 1024, BF, True), (1, 300, 4096, HF, False), (2, 64, 14336, BF, True), (5, 513, 777, HF, True),
        (16, 4096, 512, BF, False), (22, 256, 2048, HF, True), (32, 1000, 1024, BF, True), (33, 100, 100, HF, False),
        (64, 128, 256, BF, True), (100, 200, 512, HF, False), (130, 300, 1024, BF, True), (1, 1, 1, HF, True),
        (300, 1030, 1001, BF, True), (257, 513, 576, HF, True), (512, 768, 2048, BF, False), (4, 20, 16, BF, True),
        (700, 600, 640, BF, True), (1, 2050, 6000, BF, True), (8, 4000, 8200, HF, True)]


@pytest.mark.parametrize("m,n,k,dtype,bias", INT8)
def test_linear_int8(m, n, k, dtype, bias):
    x, q, s, b = _int8_case(m + n + k, m, n, k, dtype, bias)
    guard = torch.full((m + 2, n), float("nan"), dtype=dtype, device=DEV)
    bd = None if b is None else b.to(DEV)
    y = fw.linear_int8(x.to(DEV), q, s, bd, out=guard[1:-1])
    torch.cuda.synchronize()
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    ref, tol = _int8_ref(x, q, s, b)
    _assert_within(y.double().cpu().numpy(), ref, tol, f"int8 {fw.fp8w_linear_int8_kernel(m, n, k, 0, 0)}")
    qx, sx = fw.quantize_activations_int8(x.to(DEV))
    z = fw.gemm_int8(qx, sx, q, s, bd, out_dtype=dtype)
    assert torch.equal(z, y), "the two-step call differs (integer sums leave no room for it)"


@pytest.mark.parametrize("m", [1, 7, 20, 80, 300])
@pytest.mark.parametrize("qoff,xoff", [(8, 0), (1, 0), (0, 8), (0, 2), (5, 6)])
def test_linear_int8_unaligned_buffers(m, qoff, xoff):
    x, q, s, b = _int8_case(m, m, 96, 512, BF, True)
    qb = torch.empty(q.numel() + 64, dtype=torch.int8, device=DEV)
    qb[qoff:qoff + q.numel()] = q.reshape(-1)
    xb = torch.empty(x.numel() + 64, dtype=BF, device=DEV)
    xb[xoff // 2:xoff // 2 + x.numel()] = x.reshape(-1).to(DEV)
    y = fw.linear_int8(xb[xoff // 2:xoff // 2 + x.numel()].view(x.shape), qb[qoff:qoff + q.numel()].view(q.shape), s,
                       b.to(DEV))
    ref, tol = _int8_ref(x, q, s, b)
    _assert_within(y.double().cpu().numpy(), ref, tol, "unaligned int8")


@pytest.mark.parametrize("m,k", [(1, 131072), (40, 131072)])
def test_linear_int8_longest_rows_do_not_overflow(m, k):
    """All codes 127 at the largest k: the integer sum is 127 * 127 * 131072 < 2^31."""
    x = torch.ones((m, k), dtype=BF, device=DEV)
    q = torch.full((24, k), 127, dtype=torch.int8, device=DEV)
    q[1] = -127
    s = torch.full((24,), 2.0 ** -10, device=DEV)
    y = fw.linear_int8(x, q, s).double().cpu().numpy()
    ref = np.full((m, 24), 127.0 * k * 2.0 ** -10)
    ref[:, 1] *= -1
    _assert_within(y, ref, np.abs(ref) * (2.0 ** -8 + 2.0 ** -20), "longest rows")


@pytest.mark.parametrize("m", [4, 70, 300])
def test_linear_int8_zero_and_non_finite_tokens(m):
    x, q, s, b = _int8_case(m, m, 256, 512, BF, True)
    x[0] = 0.0
    x[2, 100] = float("nan")
    x[3, 511] = float("-inf")
    y = fw.linear_int8(x.to(DEV), q, s, b.to(DEV)).cpu()
    assert torch.equal(y[0], b)
    bad = ~torch.isfinite(y.float())
    assert bad[2].all() and bad[3].all() and bad.sum() == 2 * 256
    assert torch.equal(fw.linear_int8(x[:, :0].to(DEV).contiguous(), q[:, :0].contiguous(), s, b.to(DEV)).cpu(),
                       b.expand(m, -1))  # k == 0: the bias


@pytest.mark.parametrize("dtype", [FL, BF, HF])
def test_quantize_int8_weights(dtype):
    g = torch.Generator().manual_seed(3)
    w = (torch.randn((70, 333), generator=g) * 0.02).to(dtype)
    w[5] = 0.0
    q, s = fw.quantize_int8(w.to(DEV))
    amax = w.float().abs().amax(1).numpy()
    assert np.array_equal(s.cpu().numpy(), amax / np.float32(127.0))
    num = np.float32(127.0) * w.float().numpy()  # the definition's fp32 steps
    ref = np.rint(num / np.where(amax > 0, amax, np.float32(1.0))[:, None])
    assert np.array_equal(q.cpu().numpy(), ref)
    w[3, 3] = float("nan")
    with pytest.raises(fw.Fp8wMoeError) as err:
        fw.quantize_int8(w.to(DEV))
    assert err.value.status == fw.ERR_NONFINITE


# ------------------------------------------------------------------ together
def _block(x, logits, wu, wd, ws):
    r = fw.route(logits, 2)
    h = fw.linear_experts(x, *wu, r.offsets, x_rows=r.tokens)
    a = torch.nn.functional.silu(h)
    y = fw.linear_experts(a, *wd, r.offsets, y_rows=r.slots)
    return fw.combine(y, r.weights) + fw.linear_int8(x, *ws)


def _block_weights(e, n, k):
    g = torch.Generator().manual_seed(9)
    wu = fw.quantize_experts((torch.randn((e, n, k), generator=g) * 0.05).to(DEV))
    wd = fw.quantize_experts((torch.randn((e, k, n), generator=g) * 0.05).to(DEV))
    return wu, wd, fw.quantize_int8((torch.randn((k, k), generator=g) * 0.05).to(DEV))


@pytest.mark.parametrize("t", [1, 20, 400])
def test_graph_replays_equal_eager_results(t):
    e, n, k = 8, 512, 256
    weights = _block_weights(e, n, k)
    x = torch.zeros((t, k), dtype=BF, device=DEV)
    logits = torch.zeros((t, e), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _block(x, logits, *weights)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _block(x, logits, *weights)
    g = torch.Generator().manual_seed(t)
    for step in range(4):
        x.copy_(torch.randn((t, k), generator=g))
        logits.copy_(torch.randn((t, e), generator=g))
        if step == 2:
            logits[0] = float("-inf")  # a padding token
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = _block(x, logits, *weights)
        torch.cuda.synchronize()
        assert torch.equal(got, want), f"replay {step}"


def test_calls_follow_the_current_stream():
    """On a side stream behind a long copy: the calls must wait for it there."""
    e, n, k, t = 4, 256, 256, 64
    weights = _block_weights(e, n, k)
    g = torch.Generator().manual_seed(1)
    xs, ls = torch.randn((t, k), generator=g).to(BF).to(DEV), torch.randn((t, e), generator=g).to(DEV)
    want = _block(xs, ls, *weights)
    big = torch.zeros(1 << 28, device=DEV)
    x, l = torch.zeros_like(xs), torch.zeros_like(ls)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(4):
            big.add_(1.0)
        x.copy_(xs)
        l.copy_(ls)
        got = _block(x, l, *weights)
    side.synchronize()
    assert torch.equal(got, want)


def test_repeated_calls_give_the_same_bits():
    weights = _block_weights(8, 512, 256)
    g = torch.Generator().manual_seed(2)
    x, l = torch.randn((500, 256), generator=g).to(BF).to(DEV), torch.randn((500, 8), generator=g).to(DEV)
    first = _block(x, l, *weights)
    for _ in range(5):
        assert torch.equal(_block(x, l, *weights), first)
