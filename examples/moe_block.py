"""A mixture-of-experts feed-forward block on quantized weights, checked against 64 bits.

    python examples/moe_block.py [--tokens 64] [--hidden 1024] [--inner 512] [--experts 16] [--top 4] [--dtype bf16]

One block as a serving program runs it, six calls:

    r = route(logits, top)                                     each token's experts, weights and row lists
    g, u = linear_experts(x, gate and up, .., x_rows=r.tokens) gathers the tokens, rows ordered by expert
    a = silu(g) * u
    y = linear_experts(a, down, .., y_rows=r.slots)            scatters back, rows by token and choice
    out = combine(y, r.weights) + linear_int8(x, shared)       the weighted sum, and a dense shared expert

The experts' weights are e4m3 codes with a scale per output channel, the shared
expert's int8 with the activations quantized per token in the call.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_weight_only_amd as fw  # noqa: E402


class MoeBlock:
    """Quantizes once; a call runs the block on x [t, hidden] of bf16 or fp16."""

    def __init__(self, router, gate, up, down, shared, top):
        """fp32 weights: router [e, hidden], gate and up [e, inner, hidden], down [e, hidden, inner], shared
        [hidden, hidden]."""
        self.top, self.inner, self.router = top, gate.shape[1], router
        self.gate_up = fw.quantize_experts(torch.cat([gate, up], dim=1).contiguous())  # one call for both
        self.down = fw.quantize_experts(down)
        self.shared = fw.quantize_int8(shared)

    def __call__(self, x):
        r = fw.route(x.float() @ self.router.t(), self.top)
        h = fw.linear_experts(x, *self.gate_up, r.offsets, x_rows=r.tokens)
        a = torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]
        y = fw.linear_experts(a.contiguous(), *self.down, r.offsets, y_rows=r.slots)
        return fw.combine(y, r.weights) + fw.linear_int8(x, *self.shared), r


def _e4m3(q):
    """The values of e4m3 codes in fp64."""
    c = q.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(c >= 128, -mag, mag)


def reference(block, x, r):
    """(out, bound) of the block in fp64 on the quantized weights and the choices r. bound counts the roundings to
    x's type on the way, each half a step of its value (h), and their growth through what follows: the products g
    and u (h each), the activation (silu's slope is below 1.1; its own rounding and the product's, h each), the
    down products (h), the weighted sum, the shared expert and their sum (h each); twice that, for second-order
    terms and the fp32 sums."""
    h = torch.finfo(x.dtype).eps / 2
    x64 = x.double()
    t, n = x.shape
    out, bound = torch.zeros_like(x64), torch.zeros_like(x64)
    q, s = block.gate_up
    d, ds = block.down
    for e in range(q.shape[0]):
        tok, place = (r.experts == e).nonzero(as_tuple=True)
        if tok.numel() == 0:
            continue
        w = (_e4m3(q[e]) * s[e].double()[:, None]).t().contiguous()
        g, u = torch.mm(x64[tok], w).split(block.inner, dim=1)
        act = torch.nn.functional.silu(g) * u
        err = h * (1.1 * g.abs() * u.abs() + 3 * act.abs())
        w = (_e4m3(d[e]) * ds[e].double()[:, None]).t().contiguous()
        y = torch.mm(act, w)
        rw = r.weights[tok, place].double()[:, None]
        out.index_add_(0, tok, rw * y)
        bound.index_add_(0, tok, rw * (torch.mm(err, w.abs()) + h * y.abs()))
    q8, s8 = block.shared
    amax = x64.abs().amax(1, keepdim=True)
    near = 127.0 * x64 / torch.where(amax > 0, amax, 1.0)
    half = torch.floor(near) + 0.5
    codes = torch.round(torch.where((near - half).abs() < 1e-9, half, near))
    sh = torch.mm(codes, q8.double().t().contiguous()) * (amax / 127.0) * s8.double()
    bound += h * (out.abs() + sh.abs() + (out + sh).abs())
    return out + sh, 2 * bound + 1e-30


def build(hidden, inner, experts, top, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def w(*shape):
        return torch.randn(shape, generator=g, device=device) / shape[-1] ** 0.5

    return MoeBlock(w(experts, hidden), w(experts, inner, hidden), w(experts, inner, hidden),
                    w(experts, hidden, inner), w(hidden, hidden), top)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--inner", type=int, default=512)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--top", type=int, default=4)
    p.add_argument("--dtype", choices=["bf16", "fp16"], default="bf16")
    a = p.parse_args()
    block = build(a.hidden, a.inner, a.experts, a.top)
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16}[a.dtype]
    x = torch.randn((a.tokens, a.hidden), generator=torch.Generator(device="cuda").manual_seed(1),
                    device="cuda").to(dtype)
    out, r = block(x)
    want, bound = reference(block, x, r)
    worst = ((out.double() - want).abs() / bound).max().item()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        block(x)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / 20 * 1e6
    print(f"{a.tokens} tokens, {a.top} of {a.experts} experts: {us:.1f} us a block, "
          f"largest error {worst:.2f} of its bound")
    return 0 if worst <= 1 else 1


if __name__ == "__main__":
    sys.exit(main())
