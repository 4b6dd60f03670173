"""GPU parity of the products on 4-bit weights at sizes that reach every kernel and tile
of their plans, and calls as programs make them: captured, on several streams, again and
again, on weights past 32-bit offsets.

Tolerances as in the smaller tests: half a step of the output's type, and the fp32 sums'
roundings relative to the magnitudes summed (a sum that is joined from slices has no more
of them).
"""
import pytest
import torch

import fp4_util as f4
import fp8_weight_only_amd as fw
from test_gpu_fp4 import _check_linear, _dev, _experts_case, _experts_ref, _linear_case

gpu = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16

LINEAR = [
    # m, n, k, kernel
    (1, 64, 33, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (1, 1030, 1024, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (48, 130, 2048, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (3, 14400, 512, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (16, 14400, 1001, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (2, 28700, 768, "fp4_stream_kernel<CT=2,WK=1,WC=4>"),
    (5, 28700, 99, "fp4_stream_kernel<CT=2,WK=1,WC=4>"),
    (17, 28700, 33, "fp4_tile_kernel<BN=128,BM=64,W=4>"),
    (130, 28700, 70, "fp4_tile_kernel<BN=256,BM=128,W=8>"),
    (20, 100, 33, "fp4_tile_kernel<BN=64,BM=64,W=4>"),
    (33, 7200, 768, "fp4_ring_kernel<BN=64,BM=32,W=2>"),
    (9, 70, 8192, "fp4_ring_kernel<BN=64,BM=32,W=2>*8+fp4_join_kernel"),
    (1, 1, 14336, "fp4_ring_kernel<BN=64,BM=32,W=2>*16+fp4_join_kernel"),
    (257, 250, 4096, "fp4_ring_kernel<BN=64,BM=32,W=2>*4+fp4_join_kernel"),
    (65, 7200, 768, "fp4_ring_kernel<BN=128,BM=32,W=4>"),
    (33, 1030, 8192, "fp4_ring_kernel<BN=128,BM=32,W=4>*8+fp4_join_kernel"),
    (900, 1030, 768, "fp4_ring_kernel<BN=64,BM=64,W=4>"),
    (513, 61, 14336, "fp4_ring_kernel<BN=64,BM=64,W=4>*16+fp4_join_kernel"),
    (33, 28700, 768, "fp4_ring_kernel<BN=128,BM=64,W=4>"),
    (400, 4100, 256, "fp4_ring_kernel<BN=128,BM=128,W=8>"),
    (400, 4100, 384, "fp4_ring_kernel<BN=128,BM=128,W=8>"),
    (900, 4100, 256, "fp4_ring_kernel<BN=256,BM=128,W=8>"),
    (257, 28700, 256, "fp4_ring_kernel<BN=256,BM=256,W=8>"),
    (2000, 2048, 14336, "fp4_ring_kernel<BN=256,BM=256,W=8>*4+fp4_join_kernel"),
]
EXPERTS = [
    # m, e, n, k, kernel
    (3, 3, 64, 100, "fp4_stream_kernel<CT=1,WK=4,WC=1>"),
    (3, 3, 4100, 129, "fp4_stream_kernel<CT=2,WK=2,WC=2>"),
    (30, 8, 7200, 512, "fp4_stream_kernel<CT=2,WK=1,WC=4>"),
    (1030, 3, 300, 1024, "fp4_ring_kernel<BN=64,BM=32,W=2>"),
    (500, 3, 1030, 1024, "fp4_ring_kernel<BN=128,BM=32,W=4>"),
    (500, 3, 7200, 1024, "fp4_ring_kernel<BN=64,BM=64,W=4>"),
    (800, 3, 4100, 1024, "fp4_ring_kernel<BN=128,BM=64,W=4>"),
    (240, 3, 7200, 256, "fp4_ring_kernel<BN=128,BM=128,W=8>"),
    (800, 3, 4100, 256, "fp4_ring_kernel<BN=256,BM=128,W=8>"),
    (800, 3, 7200, 256, "fp4_ring_kernel<BN=256,BM=256,W=8>"),
    (2400, 3, 300, 100, "fp4_tile_kernel<BN=128,BM=32,W=4>"),
    (1300, 60, 1030, 1001, "fp4_tile_kernel<BN=128,BM=64,W=4>"),
    (800, 3, 7200, 100, "fp4_tile_kernel<BN=256,BM=128,W=8>"),
    (100, 3, 64, 129, "fp4_tile_kernel<BN=64,BM=64,W=4>"),
]
AT = 1 << 20  # any aligned address


@pytest.mark.parametrize("m,n,k,kernel", LINEAR)
def test_linear_plan(m, n, k, kernel):
    assert fw.fp8w_linear_fp4_kernel(m, n, k, AT, AT, AT) == kernel
    parts = int(kernel.split("*")[1].split("+")[0]) if "*" in kernel else 0
    assert fw.fp8w_linear_fp4_workspace_bytes(m, n, k, AT, AT, AT) == parts * m * ((n + 3) // 4 * 4) * 4


@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts_plan(m, e, n, k, kernel):
    assert fw.fp8w_linear_experts_fp4_kernel(m, e, n, k, AT, AT, AT) == kernel


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,kernel", LINEAR)
def test_linear_instance(m, n, k, kernel, dtype):
    _check_linear(*_linear_case(m + n + k, m, n, k, dtype, dtype == HF))


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,e,n,k,kernel", EXPERTS)
def test_experts_instance(m, e, n, k, kernel, dtype):
    x, q, s, b, offsets, xi, yi = _experts_case(m + n + k, m, e, n, k, dtype, dtype == HF, "even", True, True)
    out = torch.full((m, n), float("nan"), dtype=dtype, device=DEV)
    fw.linear_experts_fp4(x, q, s, _dev(offsets), b, x_rows=_dev(xi), y_rows=_dev(yi), out=out)
    ref, mag = _experts_ref(x, q, s, b, offsets, xi, yi, m)
    f4.assert_within(out, ref, f4.tolerance(ref, mag, k, dtype), kernel)


CALLS = [(1, 96, 512), (4, 4100, 640), (40, 260, 4096), (20, 100, 333), (257, 250, 4096)]


@gpu
@pytest.mark.parametrize("m,n,k", CALLS)
def test_linear_in_graphs_and_again(m, n, k):
    """Two graphs on one workspace, replayed on other values with eager calls between them."""
    x, q, s, b = _linear_case(m + k, m, n, k, BF, True)
    ws = torch.empty(max(16, fw.fp4_workspace_bytes(x, q, s)), dtype=torch.uint8, device=DEV)
    fw.linear_fp4(x, q, s, b, workspace=ws)
    torch.cuda.synchronize()
    outs, graphs = [], []
    for _ in range(2):
        out, graph = torch.empty((m, n), dtype=BF, device=DEV), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fw.linear_fp4(x, q, s, b, out=out, workspace=ws)
        outs.append(out)
        graphs.append(graph)
    for i in range(5):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV))
        want = fw.linear_fp4(x, q, s, b)
        assert torch.equal(fw.linear_fp4(x, q, s, b), want)
        for out, graph in zip(outs, graphs):
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@gpu
@pytest.mark.parametrize("m,n,k", CALLS)
def test_linear_on_streams_at_once(m, n, k):
    x, q, s, b = _linear_case(m + k, m, n, k, HF, True)
    want = fw.linear_fp4(x, q, s, b)
    torch.cuda.synchronize()
    outs = []
    for stream in [torch.cuda.Stream() for _ in range(4)] * 3:
        with torch.cuda.stream(stream):
            outs.append(fw.linear_fp4(x, q, s, b))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@gpu
@pytest.mark.parametrize("m", [1, 40])
def test_linear_weights_past_32_bits(m):
    """5 GiB of codes: the last channels are those of a small layer of the same rows."""
    n, k = (1 << 20) + 1000, 10240
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    s = torch.randint(120, 124, (n, k // 32), dtype=torch.uint8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    x = torch.randn((m, k), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(BF)
    out = fw.linear_fp4(x, q, s)
    for lo in (0, (1 << 32) // (k // 2) - 8, n - 64):
        ref, mag = f4.product(x, f4.decode(q[lo:lo + 64], s[lo:lo + 64], k, BF), None)
        f4.assert_within(out[:, lo:lo + 64], ref, f4.tolerance(ref, mag, k, BF), f"channels from {lo}")


@gpu
@pytest.mark.parametrize("rows", [2, 60])
def test_experts_weights_past_32_bits(rows):
    e, n, k = 80, 14336, 8192
    q = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    s = torch.randint(120, 124, (e, n, k // 32), dtype=torch.uint8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    x = torch.randn((2 * rows, k), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(BF)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[74:] = rows
    offsets[e] = 2 * rows
    out = fw.linear_experts_fp4(x, q, s, offsets)
    for i, r in ((73, slice(0, rows)), (e - 1, slice(rows, 2 * rows))):
        ref, mag = f4.product(x[r], f4.decode(q[i, -200:], s[i, -200:], k, BF), None)
        f4.assert_within(out[r, -200:], ref, f4.tolerance(ref, mag, k, BF), f"expert {i}")
