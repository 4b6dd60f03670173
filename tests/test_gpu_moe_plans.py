"""GPU parity of the mixture-of-experts and int8 products at sizes that reach
every kernel and tile of their plans, against plain 64-bit computations.

Tolerances count roundings as in the smaller tests: half a step of the output's
type, and the fp32 sums' roundings relative to the magnitudes summed.
"""
import numpy as np
import pytest
import torch

import fp8_weight_only_amd as fw

gpu = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25}

EXPERTS = [
    # m, e, n, k, kernel
    (1200, 4, 4096, 320, "experts_ring_kernel<BN=256,BM=256,W=8>"),
    (1030, 3, 8000, 320, "experts_ring_kernel<BN=256,BM=256,W=8>"),
    (800, 8, 7168, 384, "experts_ring_kernel<BN=256,BM=128,W=8>"),
    (800, 8, 4096, 448, "experts_ring_kernel<BN=128,BM=128,W=8>"),
    (240, 8, 7200, 320, "experts_ring_kernel<BN=256,BM=64,W=8>"),
    (240, 8, 4000, 320, "experts_ring_kernel<BN=128,BM=64,W=4>"),
    (240, 8, 2000, 576, "experts_ring_kernel<BN=64,BM=64,W=4>"),
    (40, 8, 7168, 2048, "experts_ring_kernel<BN=256,BM=32,W=4>"),
    (40, 8, 4096, 512, "experts_ring_kernel<BN=128,BM=32,W=4>"),
    (40, 8, 2000, 448, "experts_ring_kernel<BN=64,BM=32,W=2>"),
    (900, 300, 520, 384, "experts_ring_kernel<BN=128,BM=32,W=4>"),
    (200, 13, 5000, 256, "experts_tile_kernel<BN=128,BM=32,W=4>"),
    (100, 7, 6000, 129, "experts_tile_kernel<BN=128,BM=32,W=4>"),
    (500, 8, 4000, 998, "experts_tile_kernel<BN=128,BM=64,W=4>"),
    (800, 8, 7168, 257, "experts_tile_kernel<BN=256,BM=128,W=8>"),
    (560, 8, 3700, 300, "experts_tile_kernel<BN=128,BM=64,W=4>"),
    (800, 8, 1000, 77, "experts_tile_kernel<BN=64,BM=64,W=4>"),
    (3, 8, 512, 512, "experts_stream_kernel<CT=1,W=4>"),
    (3, 8, 512, 4096, "experts_stream_kernel<CT=1,W=8>"),
    (30, 16, 4096, 512, "experts_stream_kernel<CT=4,W=4>"),
    (2, 2, 14000, 2048, "experts_stream_kernel<CT=4,W=8>"),
    (40, 8, 1000, 1001, "experts_stream_kernel<CT=2,W=4>"),
    (300, 5, 256, 5000, "experts_stream_kernel<CT=1,W=8>"),
    (3, 4, 2000, 100, "experts_stream_kernel<CT=1,W=4>"),
    (2, 2, 5000, 3000, "experts_stream_kernel<CT=2,W=8>"),
]

INT8 = [
    # m, n, k, kernel (behind the quantizer's)
    (4000, 4100, 512, "int8_ring_kernel<BN=256,BM=256,W=8,NS=4>"),
    (2048, 4096, 512, "int8_ring_kernel<BN=256,BM=128,W=8,NS=4>"),
    (1024, 4096, 1024, "int8_ring_kernel<BN=128,BM=128,W=8,NS=4>"),
    (500, 4000, 576, "int8_ring_kernel<BN=128,BM=64,W=4,NS=4>"),
    (200, 300, 1024, "int8_ring_kernel<BN=64,BM=64,W=4,NS=8>"),
    (130, 512, 8192, "int8_ring_kernel<BN=64,BM=64,W=4,NS=8>*8+int8_join_kernel"),
    (64, 1001, 2048, "int8_ring_kernel<BN=64,BM=64,W=4,NS=8>*4+int8_join_kernel"),
    (9, 200, 256, "int8_ring_kernel<BN=128,BM=64,W=4,NS=4>"),
    (3, 512, 1024, "int8_stream_kernel<RT=1,CT=1,W=4>"),
    (3, 14400, 1024, "int8_stream_kernel<RT=1,CT=2,W=4>"),
    (4, 300, 5001, "int8_stream_kernel<RT=1,CT=1,W=8>"),
    (20, 512, 1001, "int8_stream_kernel<RT=2,CT=1,W=4>"),
    (20, 14400, 2050, "int8_stream_kernel<RT=2,CT=2,W=8>"),
    (50, 600, 100, "int8_stream_kernel<RT=4,CT=1,W=4>"),
    (50, 14400, 2049, "int8_stream_kernel<RT=4,CT=2,W=8>"),
    (3000, 6000, 300, "int8_tile_kernel<BN=256,BM=256,W=8>"),
    (1500, 6000, 100, "int8_tile_kernel<BN=256,BM=128,W=8>"),
    (700, 6000, 100, "int8_tile_kernel<BN=128,BM=128,W=8>"),
    (500, 1030, 1001, "int8_tile_kernel<BN=64,BM=64,W=4>"),
    (200, 250, 1999, "int8_tile_kernel<BN=64,BM=64,W=4>*4+int8_join_kernel"),
    (70, 300, 8198, "int8_tile_kernel<BN=64,BM=64,W=4>*8+int8_join_kernel"),
    (1, 1000, 1000, "int8_stream_kernel<RT=1,CT=1,W=4,FUSED>"),
    (1, 999, 16384, "int8_stream_kernel<RT=1,CT=1,W=8,FUSED>"),
    (1, 100, 20000, "int8_stream_kernel<RT=1,CT=1,W=8>"),
]


@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts_plan_names(m, e, n, k, kernel):
    assert fw.fp8w_linear_experts_kernel(m, e, n, k, 0, 0) == kernel


@pytest.mark.parametrize("m,n,k,kernel", INT8)
def test_int8_plan_names(m, n, k, kernel):
    assert fw.fp8w_linear_int8_kernel(m, n, k, 0, 0).split("+", "FUSED" not in kernel)[-1] == kernel


def _values():
    """The 256 e4m3 codes in fp64."""
    c = torch.arange(256, device="cuda")
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(c >= 128, -mag, mag)


def _within(y, ref, tol, what):
    y = y.double()
    assert torch.isfinite(y).all(), f"{what}: non-finite outputs"
    bad = ((y - ref).abs() > tol).nonzero()
    assert len(bad) == 0, f"{what}: {len(bad)} of {ref.numel()} outside, first at {bad[0].tolist()}"


@gpu
@pytest.mark.parametrize("dtype,bias,gather", [(BF, True, True), (HF, False, False)])
@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts_plans(m, e, n, k, kernel, dtype, bias, gather):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    w = 0.02 * torch.randn((e, n, k), generator=g, device="cuda")
    q, s = fw.quantize_experts(w)
    xr = max(1, m // 2) if gather else m
    x = torch.randn((xr, k), generator=g, device="cuda").to(dtype)
    b = torch.randn((e, n), generator=g, device="cuda").to(dtype) if bias else None
    lens = np.random.default_rng(m).multinomial(m - m // 16, np.random.default_rng(k).dirichlet(np.full(e, 2.0)))
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = torch.randint(0, xr, (m,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    places = None if gather else torch.randperm(m, generator=g, device="cuda").int()
    guard = torch.full((m + 2, n), float("nan"), dtype=dtype, device="cuda")
    y = fw.linear_experts(x, q, s, torch.from_numpy(offsets).cuda(), b, rows, places, out=guard[1:-1])
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    src = torch.arange(m, device="cuda") if rows is None else rows.long()
    dst = torch.arange(m, device="cuda") if places is None else places.long()
    ref = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    value = _values()
    for i in range(e):
        lo, hi = int(offsets[i]), int(offsets[i + 1])
        if hi == lo:
            continue
        wi = value[q[i].long()].t().contiguous()
        xi = x[src[lo:hi]].double()
        r, a = torch.mm(xi, wi) * s[i].double(), torch.mm(xi.abs(), wi.abs()) * s[i].double()
        if b is not None:
            r, a = r + b[i].double(), a + b[i].double().abs()
        ref[dst[lo:hi]], mag[dst[lo:hi]] = r, a
    half = torch.finfo(dtype).eps / 2
    tol = ref.abs() * half * (1 + 2.0 ** -8) + mag * (k + 8) * 2.0 ** -23 + TINY[dtype]
    _within(y, ref, tol, kernel)
    assert torch.equal(y, fw.linear_experts(x, q, s, torch.from_numpy(offsets).cuda(), b, rows, places)), "other bits"


@gpu
@pytest.mark.parametrize("dtype,bias", [(BF, True), (HF, False)])
@pytest.mark.parametrize("m,n,k,kernel", INT8)
def test_int8_plans(m, n, k, kernel, dtype, bias):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    q = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand((n,), generator=g, device="cuda") * 1e-3
    x = torch.randn((m, k), generator=g, device="cuda").to(dtype)
    b = torch.randn((n,), generator=g, device="cuda").to(dtype) if bias else None
    guard = torch.full((m + 2, n), float("nan"), dtype=dtype, device="cuda")
    y = fw.linear_int8(x, q, s, b, out=guard[1:-1])
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all(), "wrote outside the output"
    x64 = x.double()
    amax = x64.abs().amax(1, keepdim=True)
    r = 127.0 * x64 / amax
    h = torch.floor(r) + 0.5
    codes = torch.round(torch.where((r - h).abs() < 1e-9, h, r))
    prod = torch.mm(codes, q.double().t().contiguous()) * (amax / 127.0) * s.double()
    ref = prod if b is None else prod + b.double()
    # the sum to fp32, the token scale, its product, the fused multiply-add's: within five fp32 roundings
    tol = ref.abs() * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -8) + prod.abs() * 5 * 2.0 ** -24 + TINY[dtype]
    _within(y, ref, tol, kernel)
    qx, sx = fw.quantize_activations_int8(x)
    assert torch.equal(fw.gemm_int8(qx, sx, q, s, b, out_dtype=dtype), y), "the two-step call differs"


@gpu
@pytest.mark.parametrize("t,e,top", [(32, 256, 8), (33, 64, 4), (64, 128, 8), (65, 128, 8), (256, 16, 2), (257, 16, 2),
                                     (4097, 512, 3), (9000, 1024, 2), (20000, 31, 16), (8193, 33, 1), (3000, 64, 20)])
def test_route_plans(t, e, top):
    """Both sides of the single launch, of the lanes per token and of every width; ties everywhere."""
    g = torch.Generator(device="cuda").manual_seed(t + e)
    logits = torch.randint(-20, 20, (t, e), generator=g, device="cuda").float() / 4
    logits[torch.rand((t, e), generator=g, device="cuda") < 0.2] = float("-inf")
    logits[::11] = float("-inf")
    r = fw.route(logits, top)
    order = torch.sort(logits.cpu(), dim=1, descending=True, stable=True)
    ids = torch.where(torch.isinf(order.values[:, :top]), -1, order.indices[:, :top])
    assert torch.equal(r.experts.cpu().long(), ids)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, e, flat)
    slots = torch.sort(key, stable=True).indices
    assert torch.equal(r.slots.cpu().long(), slots)
    assert torch.equal(r.tokens.cpu().long(), slots // top)
    assert torch.equal(r.offsets.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long),
                                                          torch.bincount(key, minlength=e + 1)[:e].cumsum(0)]))
    v = order.values[:, :top].double()
    p = torch.where(ids < 0, 0.0, torch.exp(v - torch.where(torch.isinf(v[:, :1]), 0.0, v[:, :1])))
    ref = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    # exp of exact differences: its own two steps; the sum's top roundings; the quotient
    assert ((r.weights.cpu().double() - ref).abs() <= ref * (top + 16) * 2.0 ** -24).all()
