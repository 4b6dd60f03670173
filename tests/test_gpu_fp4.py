"""GPU parity of the 4-bit weights: quantizer and decoder bit for bit, the linear
layer and the products grouped by expert against 64-bit computations."""
import numpy as np
import pytest
import torch

import fp4_util as f4
import fp8_weight_only_amd as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", [FL, BF, HF])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 32), (5, 33), (64, 4096), (17, 1001), (2, 31), (300, 64), (1, 70000)])
def test_quantize(n, k, dtype):
    rng = np.random.default_rng(n + k)
    w = rng.standard_normal((n, k)) * np.exp2(rng.integers(-12, 12, (n, 1)))
    w[rng.random((n, k)) < 0.1] = 0.0
    w = torch.from_numpy(w).to(dtype)
    q, s = fw.quantize_fp4(w.to(DEV))
    qr, sr = f4.quantize(w.double().numpy())
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)


def test_quantize_ties_limits_and_subnormals():
    """Every half-way point, values beyond 6, blocks of zeros, the largest and smallest fp32 values."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, 4.0, 0.2499999, 0.2500001, 5.0000005, 4.9999995, -0.0])
    block = np.concatenate([ties, -ties])
    rows = [block * 2.0 ** e for e in (0, 1, -9, 100, -100, 124, -120, -126, -130, -140, -146)]
    w = np.stack(rows + [np.zeros(32), np.full(32, 3.4028235e38), np.full(32, -1e-45), np.full(32, 2.0 ** -125)])
    w = w.astype(np.float32)
    q, s = fw.quantize_fp4(torch.from_numpy(w).to(DEV))
    qr, sr = f4.quantize(w.astype(np.float64))
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_non_finite(bad):
    w = torch.ones((4, 96), device=DEV)
    w[2, 40] = bad
    with pytest.raises(fw.Fp8wMoeError) as err:
        fw.quantize_fp4(w)
    assert err.value.status == fw.ERR_NONFINITE


def test_quantize_stack_is_quantize_of_its_rows():
    w = torch.randn((3, 20, 77), device=DEV)
    q, s = fw.quantize_fp4(w)
    q2, s2 = fw.quantize_fp4(w.view(60, 77))
    assert q.shape == (3, 20, 39) and s.shape == (3, 20, 3)
    assert torch.equal(q.view(60, 39), q2) and torch.equal(s.view(60, 3), s2)


@pytest.mark.parametrize("dtype", [FL, BF, HF])
def test_dequantize_every_code_and_scale(dtype):
    """16 codes by 255 scales; an odd k leaves out the last byte's high bits."""
    s = torch.arange(255, device=DEV, dtype=torch.uint8)[:, None]
    q = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe], dtype=torch.uint8, device=DEV).expand(255, -1)
    for k in (16, 15):
        w = fw.dequantize_fp4(q.contiguous(), s, k, dtype)
        want = f4.decode(q, s, k).to(dtype)
        assert torch.equal(w.view(torch.int32 if dtype == FL else torch.int16),
                           want.view(torch.int32 if dtype == FL else torch.int16))
    nan = fw.dequantize_fp4(q[:1].contiguous(), torch.full((1, 1), 255, dtype=torch.uint8, device=DEV), dtype=dtype)
    assert torch.isnan(nan).all()


# ------------------------------------------------------------------ linear
def _linear_case(seed, m, n, k, dtype, bias, std=0.02):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, s = fw.quantize_fp4(std * torch.randn((n, k), generator=g, device=DEV))
    x = torch.randn((m, k), generator=g, device=DEV).to(dtype)
    b = torch.randn((n,), generator=g, device=DEV).to(dtype) if bias else None
    return x, q, s, b


def _check_linear(x, q, s, b, what=""):
    m, k = x.shape
    n = q.shape[0]
    guard = torch.full((m + 2, n), float("nan"), dtype=x.dtype, device=DEV)
    fw.linear_fp4(x, q, s, b, out=guard[1:-1])
    torch.cuda.synchronize()
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    ref, mag = f4.product(x, f4.decode(q, s, k, x.dtype), b)
    name = fw.fp8w_linear_fp4_kernel(m, n, k, x.data_ptr(), q.data_ptr(), s.data_ptr())
    f4.assert_within(guard[1:-1], ref, f4.tolerance(ref, mag, k, x.dtype), f"{what} m={m} n={n} k={k} {name}")


LINEAR = [(1, 1, 1), (1, 1024, 1024), (1, 300, 4096), (2, 33, 77), (5, 40, 17), (16, 256, 256), (17, 520, 512),
          (1, 16, 8192), (22, 130, 1999), (32, 96, 640), (33, 64, 2048), (64, 257, 1001), (65, 200, 320),
          (100, 130, 77), (129, 64, 64), (130, 1030, 1002), (300, 264, 512), (333, 257, 384), (700, 200, 1000),
          (1500, 768, 256), (40, 512, 32), (3, 70, 31), (9, 128, 96), (2, 100, 260), (70, 100, 33)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(m, n, k, dtype, bias):
    _check_linear(*_linear_case(m + n + k, m, n, k, dtype, bias))


@pytest.mark.parametrize("m", [1, 3, 20, 90, 600])
@pytest.mark.parametrize("qoff,soff,xoff", [(8, 0, 0), (1, 0, 0), (0, 1, 0), (0, 2, 0), (0, 0, 8), (0, 0, 2), (3, 3, 6)])
def test_linear_unaligned_buffers(m, qoff, soff, xoff):
    x, q, s, b = _linear_case(m, m, 96, 512, BF, True)

    def moved(t, off):
        buf = torch.full((t.numel() + 64,), 0x55, dtype=t.dtype, device=DEV)
        off //= t.element_size()
        buf[off:off + t.numel()] = t.reshape(-1)
        return buf[off:off + t.numel()].view(t.shape)
    _check_linear(moved(x, xoff), moved(q, qoff), moved(s, soff), b)


@pytest.mark.parametrize("m,k", [(1, 33), (1, 301), (40, 65), (300, 129), (20, 511)])
def test_linear_ignores_the_spare_bits_of_odd_rows(m, k):
    x, q, s, b = _linear_case(k, m, 70, k, HF, True)
    want = fw.linear_fp4(x, q, s, b)
    q[:, -1] |= 0x70
    assert torch.equal(fw.linear_fp4(x, q, s, b), want)


@pytest.mark.parametrize("m", [1, 20, 200])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_over_the_range_of_scales(m, dtype):
    """Rows of one scale each: those whose weights and sums are the type's finite values."""
    lo, hi = (-100, 100) if dtype == BF else (-23, 6)
    n, k = hi - lo + 1, 512
    g = torch.Generator(device=DEV).manual_seed(m)
    q = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (torch.arange(lo, hi + 1, device=DEV) + 127).to(torch.uint8)[:, None].expand(n, k // 32).contiguous()
    x = torch.randn((m, k), generator=g, device=DEV).to(dtype)
    _check_linear(x, q, s, None)


def test_linear_fp16_weights_past_the_type():
    """Below 2^-23 a weight rounds to fp16's subnormals, above 65504 it is infinite."""
    x = torch.zeros((1, 32), dtype=HF, device=DEV)
    x[0, 0] = 1.0
    q = torch.full((3, 16), 0x07, dtype=torch.uint8, device=DEV)  # 6 at even k
    s = torch.tensor([[127 + 14], [127 - 25], [127 - 28]], dtype=torch.uint8, device=DEV)
    y = fw.linear_fp4(x, q, s)
    assert torch.isnan(y[0, 0])  # an infinite weight times 0 at the other k
    assert y[0, 1:].view(torch.int16).cpu().tolist() == [3, 0]
    y = fw.linear_fp4(torch.ones_like(x), q, s)
    assert y[0, 0] == float("inf") and y[0, 1:].view(torch.int16).cpu().tolist() == [48, 0]


@pytest.mark.parametrize("m", [2, 40, 200])
def test_linear_nan_and_infinity_stay_in_their_rows(m):
    x, q, s, b = _linear_case(m, m, 96, 512, BF, True)
    want = fw.linear_fp4(x, q, s, b)
    x[1, 5] = float("nan")
    y = fw.linear_fp4(x, q, s, b)
    assert torch.isnan(y[1]).all() and torch.equal(y[torch.arange(m) != 1], want[torch.arange(m) != 1])
    s[7, 3] = 255  # a scale of NaN: that channel
    y = fw.linear_fp4(x, q, s, b)
    assert torch.isnan(y[:, 7]).all() and torch.isnan(y[0]).sum() == 1


def test_linear_no_tokens_no_width_no_channels():
    x, q, s, b = _linear_case(1, 3, 16, 64, BF, True)
    assert fw.linear_fp4(x[:0], q, s, b).shape == (0, 16)
    assert fw.linear_fp4(x, q[:0], s[:0], b[:0]).shape == (3, 0)
    none = torch.empty((16, 0), dtype=torch.uint8, device=DEV)
    assert torch.equal(fw.linear_fp4(x[:, :0].contiguous(), none, none, b), b.expand(3, -1))


# ------------------------------------------------------------------ experts
def _lengths(rng, m, e, kind):
    """Ragged group sizes with sum <= m."""
    if kind == "one":
        n = np.zeros(e, dtype=int)
        n[e // 2] = m
        return n
    n = rng.multinomial(m, rng.dirichlet(np.full(e, 0.3 if kind == "skew" else 5.0)))
    if kind == "tail":
        n[-1] = 0
        n = n // 2
    return n


def _experts_case(seed, m, e, n, k, dtype, bias, kind, gather, scatter):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, s = fw.quantize_fp4(0.02 * torch.randn((e, n, k), generator=g, device=DEV))
    xr = max(1, m // 2) if gather else m
    x = torch.randn((xr, k), generator=g, device=DEV).to(dtype)
    b = torch.randn((e, n), generator=g, device=DEV).to(dtype) if bias else None
    offsets = np.concatenate([[0], np.cumsum(_lengths(rng, m, e, kind))]).astype(np.int32)
    xi = rng.integers(0, xr, m).astype(np.int32) if gather else None
    yi = rng.permutation(m).astype(np.int32) if scatter else None
    return x, q, s, b, offsets, xi, yi


def _dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def _experts_ref(x, q, s, b, offsets, xi, yi, m):
    e, n = q.shape[:2]
    k = x.shape[1]
    y = torch.zeros((m, n), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    for i in range(e):
        p = np.arange(offsets[i], offsets[i + 1])
        if len(p) == 0:
            continue
        src, dst = _dev(p if xi is None else xi[p].astype(np.int64)), _dev(p if yi is None else yi[p].astype(np.int64))
        y[dst], mag[dst] = f4.product(x[src], f4.decode(q[i], s[i], k, x.dtype), None if b is None else b[i])
    return y, mag


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
    x, q, s, b, offsets, xi, yi = _experts_case(m + n, m, e, n, k, dtype, bias, kind, gather, scatter)
    guard = torch.full((m + 2, n), float("nan"), dtype=dtype, device=DEV)
    fw.linear_experts_fp4(x, q, s, _dev(offsets), b, _dev(xi), _dev(yi), out=guard[1:-1])
    torch.cuda.synchronize()
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    ref, mag = _experts_ref(x, q, s, b, offsets, xi, yi, m)
    f4.assert_within(guard[1:-1], ref, f4.tolerance(ref, mag, k, dtype),
                     f"m={m} e={e} n={n} k={k} {fw.fp8w_linear_experts_fp4_kernel(m, e, n, k, 0, 0, 0)}")


@pytest.mark.parametrize("m,n,k", [(6, 64, 512), (200, 128, 256), (40, 33, 100), (900, 96, 384)])
def test_linear_experts_bad_rows_and_offsets(m, n, k):
    """Device values out of range: rows of NaN, rows not written, offsets clamped; no byte outside the buffers."""
    x, q, s, b, offsets, xi, yi = _experts_case(m, m, 4, n, k, BF, False, "even", True, True)
    xi[1], xi[m - 1], yi_bad = 1 << 30, -1, yi.copy()
    lost = yi[2]
    yi_bad[2], yi_bad[0] = -5, m
    guard = torch.full((m + 2, n), 7.0, dtype=BF, device=DEV)
    fw.linear_experts_fp4(x, q, s, _dev(offsets), b, _dev(xi), _dev(yi_bad), out=guard[1:-1])
    y = guard[1:-1].float().cpu().numpy()
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    assert np.isnan(y[yi[1]]).all() and np.isnan(y[yi[m - 1]]).all()
    assert (y[lost] == 7).all() and (y[yi[0]] == 7).all()
    wild = np.array([-9, 1 << 30, 2, m + 50, -(1 << 31)], dtype=np.int32)
    guard.fill_(7.0)
    fw.linear_experts_fp4(x, q, s, _dev(wild), None, _dev(xi), None, out=guard[1:-1])
    torch.cuda.synchronize()
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()


def test_linear_experts_no_rows_no_width():
    x, q, s, b, offsets, _, _ = _experts_case(1, 4, 3, 16, 32, BF, True, "even", False, False)
    empty = torch.empty((3, 16, 0), dtype=torch.uint8, device=DEV)
    y = fw.linear_experts_fp4(x[:, :0].contiguous(), empty, empty, _dev(offsets), b)
    for i in range(3):  # k == 0: the bias
        assert torch.equal(y[offsets[i]:offsets[i + 1]], b[i].expand(offsets[i + 1] - offsets[i], -1))
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert fw.linear_experts_fp4(x[:0], q, s, none).shape == (0, 16)
    assert (fw.linear_experts_fp4(x, q, s, none, b) == 0).all()  # every row without an expert


def test_linear_is_one_expert_with_every_row():
    for m in (4, 40, 300):
        x, q, s, b = _linear_case(m, m, 200, 640, BF, True)
        off = torch.tensor([0, m], dtype=torch.int32, device=DEV)
        ref, mag = f4.product(x, f4.decode(q, s, 640), b)
        for y in (fw.linear_fp4(x, q, s, b), fw.linear_experts_fp4(x, q[None], s[None], off, b[None])):
            f4.assert_within(y, ref, f4.tolerance(ref, mag, 640, BF), f"m={m}")
