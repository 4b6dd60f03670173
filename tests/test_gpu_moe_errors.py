"""What the mixture-of-experts and int8 calls make of HIP errors: those that an
earlier call of the thread left for its own caller, launches that fail, and
allocations that do."""
import ctypes

import pytest
import torch

import fp8_weight_only_amd as fw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NO_DEVICE = 1 << 20


@pytest.fixture
def hip():
    torch.cuda.init()
    lib = ctypes.CDLL("libamdhip64.so.7")  # the one in the process
    lib.hipStreamCreate.argtypes = lib.hipStreamDestroy.argtypes = lib.hipStreamSynchronize.argtypes = [ctypes.c_void_p]
    lib.hipStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.hipStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    yield lib
    lib.hipGetLastError()


def _calls():
    """name -> (a call through the C entry, its outputs), everything allocated."""
    def zeros(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    g = torch.Generator(device="cuda").manual_seed(0)
    t, e, top, n, k = 3000, 16, 2, 96, 256
    logits = torch.randn((t, e), generator=g, device="cuda")
    w, ex, off, sl, tok = zeros(t, top, dtype=torch.float32), zeros(t, top), zeros(e + 1), zeros(t * top), zeros(t * top)
    need = fw.fp8w_route_workspace_bytes(t, e, top)
    assert need > 0  # two launches
    ws = zeros(need // 4)
    y = torch.randn((64 * top, n), generator=g, device="cuda").to(BF)
    cw, co = torch.rand((64, top), generator=g, device="cuda"), zeros(64, n, dtype=BF)
    x = torch.randn((64, k), generator=g, device="cuda").to(BF)
    q8 = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    s8, qx, sx = torch.rand((n,), generator=g, device="cuda"), zeros(64, k, dtype=torch.int8), zeros(64, dtype=torch.float32)
    y8, z8 = zeros(64, n, dtype=BF), zeros(64, n, dtype=BF)
    ws8 = zeros(fw.fp8w_linear_int8_workspace_bytes(64, n, k, x.data_ptr(), q8.data_ptr()), dtype=torch.uint8)
    qe = torch.randint(0, 120, (4, n, k), generator=g, device="cuda", dtype=torch.uint8)
    se, oe = torch.rand((4, n), generator=g, device="cuda"), torch.tensor([0, 9, 20, 20, 64], device="cuda").int()
    ye = zeros(64, n, dtype=BF)
    stream = torch.cuda.current_stream().cuda_stream
    p = torch.Tensor.data_ptr
    keep = [logits, ws, y, cw, x, q8, s8, ws8, qe, se, oe]
    return keep, {
        "route": (lambda: fw.fp8w_route(p(logits), fw.FP32, t, e, top, 1, p(w), p(ex), p(off), p(sl), p(tok), p(ws), need,
                                        stream), [w, ex, off, sl, tok]),
        "combine": (lambda: fw.fp8w_combine(p(y), fw.BF16, p(cw), 64, top, n, p(co), stream), [co]),
        "experts": (lambda: fw.fp8w_linear_experts(p(x), fw.BF16, 64, k, p(qe), p(se), 0, 4, n, p(oe), 64, 0, 0, p(ye), 0,
                                                   0, stream), [ye]),
        "quantize": (lambda: fw.fp8w_quantize_activations_int8(p(x), fw.BF16, 64, k, p(qx), p(sx), stream), [qx, sx]),
        "gemm": (lambda: fw.fp8w_gemm_int8(p(qx), p(sx), 64, k, p(q8), p(s8), 0, n, p(z8), fw.BF16, stream), [z8]),
        "linear": (lambda: fw.fp8w_linear_int8(p(x), fw.BF16, 64, k, p(q8), p(s8), 0, n, p(y8), p(ws8), ws8.numel(),
                                               stream), [y8]),
        "weights": (lambda: fw.fp8w_quantize_int8(p(x), fw.BF16, 64, k, p(qx), p(sx), stream), [qx, sx]),
    }


def test_an_error_left_by_an_earlier_call_is_not_the_launch_s(hip):
    """A call neither fails for it nor takes it from its owner."""
    keep, calls = _calls()
    want = {}
    for name, (call, outs) in calls.items():
        assert call() == fw.SUCCESS
        torch.cuda.synchronize()
        want[name] = [o.clone() for o in outs]
    for name, (call, outs) in calls.items():
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    for name, (call, outs) in calls.items():
        hip.hipGetLastError()
        left = hip.hipSetDevice(NO_DEVICE)
        assert left != 0 and hip.hipPeekAtLastError() == left
        status = call()
        after = hip.hipGetLastError()
        torch.cuda.synchronize()
        assert status == fw.SUCCESS, name
        assert after == left, f"{name}: the error was taken from its owner"
        assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name


def test_a_failed_launch_is_raised_and_not_tried_again(hip, monkeypatch):
    """A launch into a capture that has become invalid is refused by HIP."""
    y, w = torch.ones((6, 40), dtype=BF, device="cuda"), torch.full((3, 2), 0.5, device="cuda")
    out = torch.zeros((3, 40), dtype=BF, device="cuda")
    again = []
    entry = fw.moe.fp8w_combine
    monkeypatch.setattr(fw.moe, "fp8w_combine", lambda *a: again.append(a) or entry(*a))
    torch.cuda.synchronize()
    own = ctypes.c_void_p()  # not one of torch's pool: it stays invalid
    assert hip.hipStreamCreate(ctypes.byref(own)) == 0
    try:
        assert hip.hipStreamBeginCapture(own, 2) == 0
        assert hip.hipStreamSynchronize(own) != 0  # not allowed while capturing: the capture is invalid
        with torch.cuda.stream(torch.cuda.ExternalStream(own.value)):
            with pytest.raises(fw.Fp8wMoeError) as err:
                fw.combine(y, w, out)
    finally:
        graph = ctypes.c_void_p()
        hip.hipStreamEndCapture(own, ctypes.byref(graph))
        hip.hipStreamDestroy(own)
        hip.hipGetLastError()
    assert err.value.status == fw.ERR_HIP and fw.fp8w_moe_last_hip_error() != 0
    assert not again, "enqueued once more"
    fw.combine(y, w, out)
    torch.cuda.synchronize()
    assert (out == 1).all()


def test_a_failed_allocation_raises_torch_s_error():
    """An output larger than the GPU's memory, through the compiled helpers as through Python."""
    m, n, k = 1 << 21, 1 << 18, 16
    x = torch.zeros((m, k), dtype=BF, device="cuda")
    q, s = torch.zeros((n, k), dtype=torch.int8, device="cuda"), torch.zeros((n,), device="cuda")
    for extra in ({}, {"workspace": torch.zeros(16, dtype=torch.uint8, device="cuda")}):
        with pytest.raises(torch.OutOfMemoryError):
            fw.linear_int8(x, q, s, **extra)
    y = fw.linear_int8(x[:64], q[:64], s[:64])
    assert (y == 0).all()
