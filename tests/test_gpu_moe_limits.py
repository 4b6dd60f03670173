"""The int8 operators at the ends of their documented sizes and codes."""
import pytest
import torch

import fp8_weight_only_amd as fw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LONGEST = 131072


@pytest.mark.parametrize("m", [1, 4, 20, 40, 70])
@pytest.mark.parametrize("off", [0, 1])
def test_gemm_int8_sum_of_the_lowest_codes(m, off):
    """-128 * -128, 131072 times, is 2^31: one more than a 32-bit integer holds. Beside it the sums next to that and
    the most negative one. The scales are powers of two; fp32 rounds the sums' neighbours of 2^31 and bf16 the results,
    so each output is a sum's bf16 value."""
    n, k = 70, LONGEST
    buf = torch.full((n * k + 16,), -128, dtype=torch.int8, device="cuda")
    q = buf[off:off + n * k].view(n, k)
    q[1] = 127
    q[2, 0] = 127
    q[3, -1] = -127
    q[4, : k // 2] = 127
    qx = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    sx = torch.full((m,), 2.0 ** -16, device="cuda")
    scale = torch.full((n,), 2.0 ** -10, device="cuda")
    bias = torch.arange(n, device="cuda").to(BF) / 4
    sums = [16384 * k] * n
    sums[1] = -16256 * k
    sums[2] -= 16384 + 16256
    sums[3] -= 128
    sums[4] = (16384 - 16256) * (k // 2)
    want = torch.tensor(sums, dtype=torch.float64).float().double() * 2.0 ** -26 + bias.cpu().double()
    y = fw.gemm_int8(qx, sx, q, scale, bias)
    assert torch.equal(y.cpu(), want.to(BF).expand(m, -1))


ROWS = (1 << 24) + 3  # 256 threads each: past the 2^32 threads of a launch


def _row_codes(x):
    """(codes, scales) by the definition; the quotient of 16-bit values, in fp64, is a half or over 1e-9 away from one."""
    x64 = x.double()
    amax = x64.abs().amax(1, keepdim=True)
    r = 127.0 * x64 / torch.where(amax > 0, amax, 1.0)
    half = torch.floor(r) + 0.5
    r = torch.where((r - half).abs() < 1e-9, half, r)
    return torch.round(r).to(torch.int8), (amax[:, 0] / 127.0).float()


def _same_codes(q, scale, x):
    for lo in range(0, x.shape[0], 1 << 22):
        part = slice(lo, lo + (1 << 22))
        codes, scales = _row_codes(x[part])
        assert torch.equal(q[part], codes) and torch.equal(scale[part], scales), lo


@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_activation_rows_past_one_launch(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((ROWS, 8), generator=g, device="cuda").to(dtype)
    _same_codes(*fw.quantize_activations_int8(x), x)


def test_weight_rows_past_one_launch():
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn((ROWS, 6), generator=g, device="cuda").to(BF)
    _same_codes(*fw.quantize_int8(w), w)
    w = w.float()
    q, s = fw.quantize_int8(w)  # fp32 rows: the other quantizer, the same values
    _same_codes(q, s, w)


def test_linear_int8_rows_past_one_launch():
    g = torch.Generator(device="cuda").manual_seed(3)
    n, k = 8, 24
    x = torch.randn((ROWS, k), generator=g, device="cuda").to(BF)
    q = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand((n,), generator=g, device="cuda") * 1e-2
    y = fw.linear_int8(x, q, s)
    for lo in range(0, ROWS, 1 << 22):
        part = slice(lo, lo + (1 << 22))
        codes, _ = _row_codes(x[part])
        amax = x[part].double().abs().amax(1, keepdim=True)
        ref = torch.mm(codes.double(), q.double().t().contiguous()) * (amax / 127.0) * s.double()
        # half a step of bf16, the fp32 scale, and the epilogue's fp32 roundings
        tol = ref.abs() * (2.0 ** -8 * (1 + 2.0 ** -8) + 5 * 2.0 ** -24) + 2.0 ** -134
        assert ((y[part].double() - ref).abs() <= tol).all(), lo
