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
