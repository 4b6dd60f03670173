"""Inputs whose sums are exact in fp32 in any order and any grouping: activations are small whole numbers, weights short
multiples of a power of two, and the magnitudes of a sum stay below 2^24 of its unit. A kernel's result then has one
rounding, that of the output's type, and is known bit for bit: a lost or doubled part of a sum, or one that passes
through fewer bits, shows in nearly every element however long the rows are.
"""
import torch

BITS = 2.0 ** 24


def whole(shape, g, dtype, most=2):
    """Whole numbers -most .. most."""
    return torch.randint(-most, most + 1, shape, generator=g, device=g.device).to(dtype)


def fp4_weights(shape, g):
    """(q, scale) of weights [.., n, k]: any codes, scales 1/2, 1 and 2, so weights are multiples of 1/4."""
    *lead, k = shape
    q = torch.randint(0, 256, (*lead, (k + 1) // 2), generator=g, device=g.device, dtype=torch.uint8)
    s = torch.randint(126, 129, (*lead, (k + 31) // 32), generator=g, device=g.device, dtype=torch.uint8)
    return q, s


def product(x, w, bias=None, unit=0.25):
    """x @ w.T + bias in fp64, after making sure that fp32 sums of it are exact."""
    y = torch.mm(x.double(), w.t().contiguous())
    mag = torch.mm(x.double().abs(), w.abs().t().contiguous())
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    assert mag.numel() == 0 or mag.max().item() < BITS * unit
    return y


def assert_bits(got, ref, what):
    """got is ref (exact in fp32) rounded once to its type."""
    want = ref.float().to(got.dtype)
    assert torch.equal(ref.float().double(), ref), "the reference itself is not exact in fp32"
    bad = (got != want).nonzero()
    assert len(bad) == 0 and torch.isfinite(got).all(), (
        f"{what}: {len(bad)} of {want.numel()} differ, first at {bad[:1].tolist()}: "
        f"{got[tuple(bad[0])].item() if len(bad) else None} against {want[tuple(bad[0])].item() if len(bad) else None}")
