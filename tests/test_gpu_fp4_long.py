"""The linear layer on 4-bit weights with activations past 2 GiB: the tiles of a long prompt, not the kernel of few
rows, which would read all the weights again for every sixteen."""
import pytest
import torch

import exact_util as ex
import fp4_util as f4
import fp8_weight_only_amd as fw

gpu = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16
AT = 1 << 20  # any aligned address


@pytest.mark.parametrize("n,k,rows", [(4096, 14336, (74898, 74899, 131072)), (1024, 4096, (262144, 262145, 1 << 20)),
                                      (14336, 4096, (262144, 262145)), (300, 1 << 20, (1024, 1025, 4096))])
def test_plan_on_both_sides(n, k, rows):
    """The last row below 2 GiB, the first behind it, and far behind."""
    assert 2 * rows[0] * k <= 1 << 31 < 2 * rows[1] * k
    for m in rows:
        assert fw.fp8w_linear_fp4_kernel(m, n, k, AT, AT, AT).startswith("fp4_ring_kernel"), m


def test_plan_of_experts_past_2_gib():
    """Gathered rows are offset from x itself."""
    assert fw.fp8w_linear_experts_fp4_kernel(262144, 8, 1024, 4096, AT, AT, AT).startswith("fp4_ring_kernel")
    assert fw.fp8w_linear_experts_fp4_kernel(262145, 8, 1024, 4096, AT, AT, AT).startswith("fp4_tile_kernel")


@gpu
@pytest.mark.parametrize("m,n,k,dtype", [((1 << 17) + 37, 4096, 8448, BF), ((1 << 17) + 37, 60, 8448, HF), (8300, 300, 1 << 17, BF)])
def test_linear_activations_past_2_gib(m, n, k, dtype):
    assert 2 * m * k > 1 << 31
    assert fw.fp8w_linear_fp4_kernel(m, n, k, AT, AT, AT).startswith("fp4_ring_kernel")
    g = torch.Generator(device=DEV).manual_seed(m + n)
    x = ex.whole((m, k), g, dtype)
    q, s = ex.fp4_weights((n, k), g)
    out = fw.linear_fp4(x, q, s)
    border = (1 << 30) // k
    for lo, hi in ((0, 40), (border - 20, border + 20), (m - 40, m)):
        ex.assert_bits(out[lo:hi], ex.product(x[lo:hi], f4.decode(q, s, k, dtype)), f"rows from {lo}")
