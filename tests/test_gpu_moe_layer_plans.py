"""GPU parity of the mixture-of-experts layer at sizes that reach each of its kernels: rows
of weights at 16-byte, 4-byte and odd boundaries, one token, up to 16 and more, second
launches that share their steps among workgroups, weights past 32-bit offsets.

The tolerance is that of the smaller tests (test_gpu_moe_layer.reference); sums that pass
through the workspace are fp32 sums like the others.
"""
import pytest
import torch

import fp4_util as f4
import fp8_weight_only_amd as fw
from test_gpu_moe_layer import check, make, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32

# hidden and inner: how a row of the first and of the second launch lies (e4m3 bytes; 4-bit ones are half as long)
ROWS = [(256, 512), (260, 520), (264, 264), (130, 130), (513, 257), (1028, 36), (64, 2000), (128, 1999), (2048, 1024)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t", [1, 7, 16, 29, 64])
@pytest.mark.parametrize("hidden,inner", ROWS)
def test_every_kernel(hidden, inner, t, fmt, dtype):
    check(make(t + hidden, fmt, t, 12, 3, hidden, inner, dtype, FL, bias=dtype == HF, masked=0.1 if t > 1 else 0.0), True,
          f"{fmt} inner={inner}")


# few output channels and many steps: eight, four and two workgroups to 16 channels
SHARED = [(16, 60, 4, 64, 2000), (1, 64, 8, 128, 4096), (64, 40, 2, 1030, 513), (40, 30, 3, 1500, 640), (5, 16, 4, 2500, 2048)]


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
@pytest.mark.parametrize("t,e,top,hidden,inner", SHARED)
def test_shared_steps(t, e, top, hidden, inner, fmt):
    check(make(t, fmt, t, e, top, hidden, inner, BF, bias=True), False, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_shared_steps_without_any(fmt):
    """More workgroups than steps, and no step at all: zeros, and the biases' sum."""
    x, l, top, up, down, ub, db = make(3, fmt, 9, 60, 4, 64, 2000, BF, bias=True)
    l[:, 1:] = float("-inf")
    check((x, l, top, up, down, ub, db))
    l[:] = float("-inf")
    assert (fw.moe_layer(x, l, top, up, down, ub, db) == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_shared_steps_again_in_graphs_and_on_streams(fmt):
    """The sums are added in one order whichever workgroup comes last: the same bits every time."""
    x, l, top, up, down, ub, db = make(4, fmt, 16, 60, 4, 200, 2000, BF, bias=True)
    want = fw.moe_layer(x, l, top, up, down, ub, db)
    for _ in range(50):
        assert torch.equal(fw.moe_layer(x, l, top, up, down, ub, db), want)
    torch.cuda.synchronize()
    outs = []
    for stream in [torch.cuda.Stream() for _ in range(4)] * 4:
        with torch.cuda.stream(stream):
            outs.append(fw.moe_layer(x, l, top, up, down, ub, db))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    ws = torch.empty(fw.moe_layer_workspace_bytes(x, l, top, up), dtype=torch.uint8, device=DEV)
    graphs = []
    for _ in range(2):
        out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fw.moe_layer(x, l, top, up, down, ub, db, out=out, workspace=ws)
        graphs.append((graph, out))
    for i in range(6):
        l.copy_(torch.randn(l.shape, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV))
        want = fw.moe_layer(x, l, top, up, down, ub, db)
        ws.fill_(0xff)  # nothing is kept from the call before
        for graph, out in graphs:
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs)


@pytest.mark.parametrize("t", [1, 10])
@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_weights_past_32_bits(fmt, t):
    e, hidden, inner = (40, 4096, 14336) if fmt == "e4m3" else (80, 4096, 14336)
    g = torch.Generator(device=DEV).manual_seed(7)

    def weights(n, k):
        if fmt == "fp4":
            return (torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device=DEV, generator=g),
                    torch.randint(118, 121, (e, n, k // 32), dtype=torch.uint8, device=DEV, generator=g))
        q = torch.randint(0, 120, (e, n, k), dtype=torch.uint8, device=DEV, generator=g)
        return q, torch.full((e, n), 2.0 ** -12, device=DEV)
    up, down = weights(2 * inner, hidden), weights(hidden, inner)
    x = (0.1 * torch.randn((t, hidden), device=DEV, generator=g)).to(BF)
    l = torch.full((t, e), -50.0, device=DEV)
    l[:, e - 1], l[:, e - 4] = 2.0, 1.0
    out = fw.moe_layer(x, l, 2, up, down)
    ref, bound = reference(x, l, 2, up, down, None, None, True)
    f4.assert_within(out, ref, bound, fmt)
