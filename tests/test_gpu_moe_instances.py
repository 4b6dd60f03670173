"""GPU parity of the instances of the int8, experts' and weighted-sum kernels
that the other tests' sizes do not select: long rows of many tokens in the int8
quantizer, k splits of the larger ring tiles, more tokens in the stream kernels,
rows below dword alignment, and row counts of the weighted sum.

Tolerances count roundings: half a step of the output's type, and the fp32 sums'
roundings relative to the magnitudes summed.
"""
import pytest
import torch

import fp8_weight_only_amd as fw
import test_gpu_moe_plans as plans

gpu = pytest.mark.gpu
BF, HF = plans.BF, plans.HF

INT8 = [
    # m, n, k, kernel (behind the quantizer's)
    (72, 2198, 5120, "int8_ring_kernel<BN=128,BM=128,W=8,NS=4>*8+int8_join_kernel"),
    (5, 4303, 6144, "int8_ring_kernel<BN=256,BM=128,W=8,NS=4>*8+int8_join_kernel"),
    (147, 12285, 11008, "int8_ring_kernel<BN=256,BM=256,W=8,NS=4>*4+int8_join_kernel"),
    (2, 14331, 1062, "int8_stream_kernel<RT=1,CT=2,W=4>"),
    (2, 14335, 2890, "int8_stream_kernel<RT=1,CT=2,W=8>"),
    (3, 14400, 2052, "int8_stream_kernel<RT=1,CT=2,W=8>"),
    (21, 256, 692, "int8_stream_kernel<RT=2,CT=1,W=4>"),
    (18, 258, 4560, "int8_stream_kernel<RT=2,CT=1,W=8>"),
    (27, 256, 2866, "int8_stream_kernel<RT=2,CT=1,W=8>"),
    (60, 257, 335, "int8_stream_kernel<RT=4,CT=1,W=4>"),
    (48, 430, 6556, "int8_stream_kernel<RT=4,CT=1,W=8>"),
    (42, 301, 2150, "int8_stream_kernel<RT=4,CT=1,W=8>"),
    (1, 257, 4121, "int8_stream_kernel<RT=1,CT=1,W=8,FUSED>"),
    (774, 5377, 262, "int8_tile_kernel<BN=128,BM=128,W=8>"),
    (669, 9918, 278, "int8_tile_kernel<BN=256,BM=128,W=8>"),
    (2046, 8959, 271, "int8_tile_kernel<BN=256,BM=256,W=8>"),
    (145, 255, 2004, "int8_tile_kernel<BN=64,BM=64,W=4>*4+int8_join_kernel"),
    (94, 383, 388, "int8_tile_kernel<BN=64,BM=64,W=4>"),
    (1030, 200, 4096, "int8_ring_kernel<BN=64,BM=64,W=4,NS=8>*2+int8_join_kernel"),  # the quantizer's long rows
    (1030, 200, 4095, "int8_tile_kernel<BN=64,BM=64,W=4>*2+int8_join_kernel"),
]

EXPERTS = [
    # m, e, n, k, kernel
    (1, 4, 256, 4926, "experts_stream_kernel<CT=1,W=8>"),
    (3, 3, 3328, 256, "experts_stream_kernel<CT=2,W=4>"),
    (2, 2, 4529, 2605, "experts_stream_kernel<CT=2,W=8>"),
    (8, 7, 2560, 326, "experts_stream_kernel<CT=4,W=4>"),
    (2, 2, 10497, 3631, "experts_stream_kernel<CT=4,W=8>"),
    (444, 3, 12543, 256, "experts_tile_kernel<BN=256,BM=128,W=8>"),
]


@pytest.mark.parametrize("m,n,k,kernel", INT8)
def test_int8_names(m, n, k, kernel):
    assert fw.fp8w_linear_int8_kernel(m, n, k, 0, 0).split("+", "FUSED" not in kernel)[-1] == kernel


@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts_names(m, e, n, k, kernel):
    assert fw.fp8w_linear_experts_kernel(m, e, n, k, 0, 0) == kernel


@gpu
@pytest.mark.parametrize("dtype,bias", [(BF, True), (HF, False)])
@pytest.mark.parametrize("m,n,k,kernel", INT8)
def test_int8(m, n, k, kernel, dtype, bias):
    plans.test_int8_plans(m, n, k, kernel, dtype, bias)


@gpu
@pytest.mark.parametrize("dtype,bias,gather", [(BF, True, True), (HF, False, False)])
@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts(m, e, n, k, kernel, dtype, bias, gather):
    plans.test_experts_plans(m, e, n, k, kernel, dtype, bias, gather)


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,k", [(1030, 2500), (1030, 2501), (1100, 4096), (1100, 4095), (1024, 8192), (1025, 5691),
                                 (1024, 14336), (1027, 10071), (1024, 16384), (1023, 8193), (9, 9563), (20, 6001)])
def test_quantized_rows(m, k, dtype):
    """Each width of the one-pass quantizer, on both sides of 1024 rows: the exact quotients' nearest integers."""
    g = torch.Generator(device="cuda").manual_seed(m + k)
    x = torch.randn((m, k), generator=g, device="cuda") * 10.0 ** torch.randint(-4, 4, (m, 1), generator=g, device="cuda")
    x = x.to(dtype)
    x[1] = 0.0
    x[2, : k - 1] = 0.0  # a row whose maximum is its last value
    x[3, 1:] = 0.0
    qx, sx = fw.quantize_activations_int8(x)
    x64 = x.double()
    amax = x64.abs().amax(1, keepdim=True)
    r = 127.0 * x64 / torch.where(amax > 0, amax, 1.0)
    half = torch.floor(r) + 0.5
    r = torch.where((r - half).abs() < 1e-9, half, r)
    assert torch.equal(qx, torch.round(r).to(torch.int8))
    assert torch.equal(sx, (amax[:, 0] / 127.0).float())  # fp64: torch divides fp32 by a scalar through its reciprocal


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("top", [1, 2, 3, 4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("n", [8, 264, 1001, 2047])
def test_combine_rows(n, top, dtype):
    t = 37
    g = torch.Generator(device="cuda").manual_seed(n + top)
    y = torch.randn((t * top, n), generator=g, device="cuda").to(dtype)
    w = torch.randn((t, top), generator=g, device="cuda")
    out = torch.full((t + 2, n), float("nan"), dtype=dtype, device="cuda")
    fw.combine(y, w, out=out[1:-1])
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all(), "wrote outside the output"
    terms = y.double().view(t, top, n) * w.double()[:, :, None]
    ref, tiny = terms.sum(1), {BF: 2.0 ** -134, HF: 2.0 ** -25}[dtype]
    tol = ref.abs() * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -8) + terms.abs().sum(1) * (top + 1) * 2.0 ** -24 + tiny
    assert ((out[1:-1].double() - ref).abs() <= tol).all()
