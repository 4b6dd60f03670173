"""Decode batches above 16 tokens whose rows the rings do not take (k not a multiple of 128, or unaligned buffers): calls
with few tiles go to the stream, which splits k over its waves, instead of walking all of k on a few CUs.

Inputs whose sums are exact (exact_util): results are compared bit for bit."""
import pytest
import torch

import exact_util as ex
import fp4_util as f4
import fp8_weight_only_amd as fw

gpu = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16
AT = 1 << 20  # any aligned address

LINEAR = [
    # m, n, k, kernel
    (16, 4096, 14330, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (17, 4096, 14330, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (22, 4096, 14330, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (22, 4096, 14272, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (64, 4096, 14330, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (128, 4096, 14330, "fp4_stream_kernel<CT=2,WK=1,WC=4>"),
    (64, 1024, 8128, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (200, 1024, 8128, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (500, 250, 14331, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (33, 1030, 1001, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    # enough tiles for most CUs, or little k: tiles
    (200, 4096, 14330, "fp4_tile_kernel<BN=64,BM=64,W=4>"),
    (17, 28672, 2050, "fp4_tile_kernel<BN=128,BM=64,W=4>"),
    (17, 512, 100, "fp4_tile_kernel<BN=64,BM=64,W=4>"),
]
EXPERTS = [
    # m, e, n, k, kernel
    (40, 2, 4096, 14330, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (512, 8, 512, 4090, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (160, 8, 512, 4090, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (68, 2, 4096, 14272, "fp4_tile_kernel<BN=64,BM=64,W=4>"),
]


@pytest.mark.parametrize("m,n,k,kernel", LINEAR)
def test_linear_plan(m, n, k, kernel):
    assert fw.fp8w_linear_fp4_kernel(m, n, k, AT, AT, AT) == kernel


@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts_plan(m, e, n, k, kernel):
    assert fw.fp8w_linear_experts_fp4_kernel(m, e, n, k, AT, AT, AT) == kernel


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,kernel", LINEAR)
def test_linear(m, n, k, kernel, dtype):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = ex.whole((m, k), g, dtype)
    q, s = ex.fp4_weights((n, k), g)
    b = ex.whole((n,), g, dtype, 60) if dtype == HF else None
    out = torch.full((m + 2, n), float("nan"), dtype=dtype, device=DEV)
    fw.linear_fp4(x, q, s, b, out=out[1:-1])
    ex.assert_bits(out[1:-1], ex.product(x, f4.decode(q, s, k, dtype), b), kernel)
    assert torch.isnan(out[0]).all() and torch.isnan(out[-1]).all()


@gpu
@pytest.mark.parametrize("off", [2, 4, 8])
@pytest.mark.parametrize("m,n,k", [(22, 1024, 8192), (48, 300, 4096)])
def test_linear_unaligned_buffers(m, n, k, off):
    """Sizes that the rings take, at addresses that they do not."""
    g = torch.Generator(device=DEV).manual_seed(off)
    x = torch.zeros(m * k + 64, dtype=BF, device=DEV)[off // 2:off // 2 + m * k].view(m, k)
    x.copy_(ex.whole((m, k), g, BF))
    codes, s = ex.fp4_weights((n, k), g)
    q = torch.zeros(codes.numel() + 64, dtype=torch.uint8, device=DEV)[off - 1:off - 1 + codes.numel()].view(codes.shape)
    q.copy_(codes)
    ex.assert_bits(fw.linear_fp4(x, q, s), ex.product(x, f4.decode(q, s, k, BF)), f"off {off}")


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts(m, e, n, k, kernel, skew, dtype):
    """Rows gathered and scattered, positions without an expert, and (skew) nearly all rows with one expert."""
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = ex.whole((m, k), g, dtype)
    q, s = ex.fp4_weights((e, n, k), g)
    b = ex.whole((e, n), g, dtype, 60)
    left = m - 3
    ends = [left - (e - 1 - i) if skew else (i + 1) * left // e for i in range(e)]
    offsets = torch.tensor([0] + ends, dtype=torch.int32, device=DEV)
    xi = torch.randperm(m, generator=g, device=DEV).int()
    yi = torch.randperm(m, generator=g, device=DEV).int()
    out = torch.full((m, n), float("nan"), dtype=dtype, device=DEV)
    fw.linear_experts_fp4(x, q, s, offsets, b, x_rows=xi, y_rows=yi, out=out)
    ref = torch.zeros((m, n), dtype=torch.float64, device=DEV)
    for i in range(e):
        p = slice(offsets[i].item(), offsets[i + 1].item())
        ref[yi[p].long()] = ex.product(x[xi[p].long()], f4.decode(q[i], s[i], k, dtype), b[i])
    ex.assert_bits(out, ref, kernel)


@gpu
def test_linear_nan_and_infinity():
    """NaN and infinity stay in their tokens."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = ex.whole((40, 4090), g, BF)
    q, s = ex.fp4_weights((1030, 4090), g)
    want = fw.linear_fp4(x, q, s)
    x[3, 100], x[21, 4089] = float("nan"), float("inf")
    out = fw.linear_fp4(x, q, s)
    rest = torch.ones(40, dtype=torch.bool, device=DEV)
    rest[[3, 21]] = False
    assert torch.equal(out[rest], want[rest]) and not torch.isfinite(out[~rest]).any() and torch.isnan(out[3]).all()
