"""4-bit weights computed apart from the library: the e2m1 / e8m0 formats from their
definition, in fp64, and the tolerances of the products.

Tolerances count roundings: half a step of the output's type, and for the fp32 sums
up to 2^-23 of the magnitudes summed per product (the matrix cores may truncate).
"""
import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(w):
    """(codes [n, (k + 1) // 2], scales [n, (k + 31) // 32]) of a finite fp64 array [n, k]."""
    n, k = w.shape
    blocks = np.pad(w, ((0, 0), (0, -k % 32))).reshape(n, -1, 32)
    amax = np.abs(blocks).max(axis=2)
    s = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2 + 127, 0)
    s = np.maximum(s, 0)
    v = blocks / np.exp2(s - 127.0)[:, :, None]
    dist = np.abs(np.abs(v)[..., None] - MAGNITUDES)  # exact: short numbers
    near = dist == dist.min(axis=-1, keepdims=True)
    code = np.where(near[..., ::2].any(axis=-1), 2 * near[..., ::2].argmax(axis=-1), near.argmax(axis=-1))
    code = (code + 8 * np.signbit(v)).reshape(n, -1)[:, :k + k % 2].astype(np.uint8)
    if k % 2:
        code[:, k:] = 0
    return code[:, 0::2] | (code[:, 1::2] << 4), s.astype(np.uint8)


def decode(q, scale, k, dtype=torch.bfloat16):
    """The weights [.., n, k] in fp64 on the codes' device, as a product with activations of ``dtype`` takes them."""
    j = torch.arange(k, device=q.device)
    c = (q[..., j // 2].long() >> (4 * (j % 2))) & 15
    mag = torch.tensor(MAGNITUDES, device=q.device)[c & 7]
    w = torch.where(c >= 8, -mag, mag) * torch.pow(2.0, scale[..., j // 32].double() - 127)
    return w if dtype == torch.bfloat16 else w.to(dtype).double()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the smallest values of a type."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}[dtype]


def product(x, w, bias=None):
    """(x @ w.T + bias, sum of the magnitudes) in fp64."""
    y = torch.mm(x.double(), w.t().contiguous())
    mag = torch.mm(x.double().abs(), w.abs().t().contiguous())
    return (y, mag) if bias is None else (y + bias.double(), mag + bias.double().abs())


def tolerance(ref, mag, k, dtype):
    return ref.abs() * half_step(dtype) * (1 + 2.0 ** -8) + mag * (k + 8) * 2.0 ** -23 + tiny(dtype)


def assert_within(y, ref, tol, what):
    y = y.double()
    assert torch.isfinite(y).all(), f"{what}: non-finite outputs"
    bad = ((y - ref).abs() > tol).nonzero()
    assert len(bad) == 0, (f"{what}: {len(bad)} of {ref.numel()} outside, first at {bad[0].tolist()}: "
                           f"{y[tuple(bad[0])].item()!r} against {ref[tuple(bad[0])].item()!r}")
