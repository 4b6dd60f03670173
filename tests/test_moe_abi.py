"""Host-side checks of include/fp8w_moe.h (no GPU needed): the library exports
what the header declares and refuses invalid arguments before it enqueues
anything, so no call here reaches a kernel launch."""
import os
import re
import subprocess

import pytest
import torch

import fp8_weight_only_amd as fw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8w_moe.h")

# fake but aligned device addresses, 2^32 bytes apart: validation must fail before they are used
A, B, C, D, E, F, G, H, I = (i << 32 for i in range(1, 10))


def declared_symbols():
    with open(HEADER) as f:
        return re.findall(r"FP8W_API\s+[\w\s\*]+?\b(fp8w_\w+)\s*\(", f.read())


def test_library_exports_what_the_header_declares():
    names = declared_symbols()
    assert sorted(names) == sorted(fw.MOE_EXPORTS)
    lib = fw.load_moe()
    for name in names:
        assert hasattr(lib, name) and name in fw.__all__, name
    out = subprocess.run(["nm", "-D", "--defined-only", fw.moe_lib_path()], capture_output=True, text=True,
                         check=True).stdout
    assert sorted(l.split()[-1] for l in out.splitlines() if " T " in l and "fp8w" in l) == sorted(names)


def _route(logits=A, dtype=fw.FP32, t=4, e=16, top=2, renorm=1, w=B, ex=C, off=D, sl=E, tok=F, ws=G, wsb=1 << 20):
    return fw.fp8w_route(logits, dtype, t, e, top, renorm, w, ex, off, sl, tok, ws, wsb, 0)


def test_route_refusals():
    for bad in [dict(dtype=3), dict(t=-1), dict(e=0), dict(e=1025), dict(top=0), dict(top=17), dict(e=512, top=65),
                dict(t=1 << 31), dict(t=1 << 30, top=4), dict(logits=0), dict(w=0), dict(ex=0), dict(off=0), dict(sl=0),
                dict(tok=0), dict(w=A + 16), dict(ex=B + 4), dict(sl=E, tok=E), dict(off=C + 8), dict(ws=E),
                dict(t=0, off=0)]:
        assert _route(**bad) == fw.ERR_INVALID_VALUE, bad
    for bad in [dict(logits=A + 2), dict(logits=A + 1, dtype=fw.BF16), dict(w=B + 2), dict(ex=C + 1), dict(off=D + 2),
                dict(sl=E + 3), dict(tok=F + 2), dict(ws=G + 2)]:
        assert _route(**bad) == fw.ERR_MISALIGNED, bad
    assert fw.fp8w_route_workspace_bytes(4, 16, 17) == 0
    assert fw.fp8w_route_workspace_bytes(-1, 16, 2) == 0
    need = fw.fp8w_route_workspace_bytes(100000, 64, 2)
    if need:
        assert _route(t=100000, e=64, wsb=need - 1) == fw.ERR_WORKSPACE
        assert _route(t=100000, e=64, ws=0, wsb=need) == fw.ERR_WORKSPACE


def _experts(x=A, act=fw.BF16, xc=8, k=256, q=B, s=C, bias=D, e=4, n=128, off=E, m=8, xr=F, yr=G, y=H, ws=0, wsb=0):
    return fw.fp8w_linear_experts(x, act, xc, k, q, s, bias, e, n, off, m, xr, yr, y, ws, wsb, 0)


def test_linear_experts_refusals():
    for bad in [dict(act=fw.FP32), dict(act=9), dict(xc=-1), dict(k=-1), dict(e=0), dict(e=1025), dict(n=-1),
                dict(m=-1), dict(xc=7, xr=0), dict(x=0), dict(q=0), dict(s=0), dict(off=0), dict(y=0), dict(y=A),
                dict(y=B + 16), dict(y=C), dict(y=D), dict(y=E), dict(y=F), dict(y=G), dict(n=1 << 31),
                dict(m=1 << 31), dict(m=1 << 30, xc=1 << 30, n=1 << 20), dict(k=(1 << 31) - 1, n=(1 << 31) - 1)]:
        assert _experts(**bad) == fw.ERR_INVALID_VALUE, bad
    for bad in [dict(x=A + 1), dict(s=C + 2), dict(bias=D + 1), dict(off=E + 2), dict(xr=F + 2), dict(yr=G + 1),
                dict(y=H + 1)]:
        assert _experts(**bad) == fw.ERR_MISALIGNED, bad
    assert _experts(m=0, xc=0, xr=0) == fw.SUCCESS and _experts(n=0) == fw.SUCCESS
    assert fw.fp8w_linear_experts_kernel(0, 4, 128, 256, 0, 0) is None
    assert fw.fp8w_linear_experts_kernel(8, 0, 128, 256, 0, 0) is None
    assert fw.fp8w_linear_experts_workspace_bytes(8, 0, 128, 256, 0, 0) == 0


def test_linear_experts_workspace_is_checked():
    for m, e, n, k in [(1, 4, 256, 8192), (8, 64, 512, 4096), (2, 8, 1024, 14336)]:
        need = fw.fp8w_linear_experts_workspace_bytes(m, e, n, k, 0, 0)
        if need:
            big = dict(m=m, xc=m, e=e, n=n, k=k, wsb=need)
            assert _experts(ws=I + 8, **big) == fw.ERR_MISALIGNED
            assert _experts(ws=A, **big) == fw.ERR_INVALID_VALUE
            assert _experts(ws=H, **big) == fw.ERR_INVALID_VALUE


def _combine(y=A, act=fw.BF16, w=B, t=4, top=2, n=64, out=C):
    return fw.fp8w_combine(y, act, w, t, top, n, out, 0)


def test_combine_refusals():
    for bad in [dict(act=fw.FP32), dict(t=-1), dict(top=-1), dict(top=65), dict(n=-1), dict(y=0), dict(w=0),
                dict(out=0), dict(out=A + 32), dict(out=B), dict(t=1 << 30, n=1 << 30)]:
        assert _combine(**bad) == fw.ERR_INVALID_VALUE, bad
    for bad in [dict(y=A + 1), dict(w=B + 2), dict(out=C + 1)]:
        assert _combine(**bad) == fw.ERR_MISALIGNED, bad
    assert _combine(t=0) == fw.SUCCESS and _combine(n=0) == fw.SUCCESS


def _int8(x=A, act=fw.BF16, m=40, k=256, q=B, s=C, bias=D, n=128, y=E, ws=F, wsb=1 << 20):
    return fw.fp8w_linear_int8(x, act, m, k, q, s, bias, n, y, ws, wsb, 0)


def test_linear_int8_refusals():
    for bad in [dict(act=fw.FP32), dict(m=-1), dict(k=-1), dict(n=-1), dict(k=131073), dict(x=0), dict(q=0), dict(s=0),
                dict(y=0), dict(y=A), dict(y=B), dict(y=C), dict(y=D), dict(m=1 << 31), dict(m=1 << 30, n=1 << 30)]:
        assert _int8(**bad) == fw.ERR_INVALID_VALUE, bad
    for bad in [dict(x=A + 1), dict(s=C + 2), dict(bias=D + 1), dict(y=E + 1)]:
        assert _int8(**bad) == fw.ERR_MISALIGNED, bad
    need = fw.fp8w_linear_int8_workspace_bytes(4096, 128, 256, 0, 0)
    assert need >= 4096 * 260
    assert _int8(m=4096, wsb=need - 1) == fw.ERR_WORKSPACE
    assert _int8(m=4096, ws=0, wsb=need) == fw.ERR_WORKSPACE
    assert _int8(m=4096, ws=F + 8, wsb=need) == fw.ERR_MISALIGNED
    assert _int8(m=4096, ws=A, wsb=need) == fw.ERR_INVALID_VALUE
    assert _int8(m=4096, ws=E, wsb=need) == fw.ERR_INVALID_VALUE
    assert _int8(m=0) == fw.SUCCESS and _int8(n=0) == fw.SUCCESS
    assert fw.fp8w_linear_int8_kernel(0, 128, 256, 0, 0) is None


def test_int8_parts_refusals():
    q = fw.fp8w_quantize_int8
    assert q(A, 7, 4, 64, B, C, 0) == fw.ERR_INVALID_VALUE
    assert q(A, fw.FP32, -1, 64, B, C, 0) == fw.ERR_INVALID_VALUE
    assert q(A, fw.FP32, 4, 131073, B, C, 0) == fw.ERR_INVALID_VALUE
    assert q(0, fw.FP32, 4, 64, B, C, 0) == fw.ERR_INVALID_VALUE
    assert q(A, fw.FP32, 4, 64, A + 16, C, 0) == fw.ERR_INVALID_VALUE
    assert q(A, fw.FP32, 4, 64, B, B, 0) == fw.ERR_INVALID_VALUE
    assert q(A + 2, fw.FP32, 4, 64, B, C, 0) == fw.ERR_MISALIGNED
    assert q(A, fw.FP32, 4, 64, B, C + 2, 0) == fw.ERR_MISALIGNED
    assert q(0, fw.FP32, 0, 64, 0, 0, 0) == fw.SUCCESS
    a = fw.fp8w_quantize_activations_int8
    assert a(A, fw.FP32, 4, 64, B, C, 0) == fw.ERR_INVALID_VALUE
    assert a(A, fw.BF16, 4, 64, 0, C, 0) == fw.ERR_INVALID_VALUE
    assert a(A, fw.BF16, 4, 64, A, C, 0) == fw.ERR_INVALID_VALUE
    assert a(A + 1, fw.BF16, 4, 64, B, C, 0) == fw.ERR_MISALIGNED
    assert a(0, fw.BF16, 0, 64, 0, 0, 0) == fw.SUCCESS
    g = fw.fp8w_gemm_int8
    assert g(A, B, 4, 64, C, D, 0, 8, E, fw.FP32, 0) == fw.ERR_INVALID_VALUE
    assert g(A, 0, 4, 64, C, D, 0, 8, E, fw.BF16, 0) == fw.ERR_INVALID_VALUE
    assert g(A, B, 4, 64, C, D, 0, 8, A, fw.BF16, 0) == fw.ERR_INVALID_VALUE
    assert g(A, B + 1, 4, 64, C, D, 0, 8, E, fw.BF16, 0) == fw.ERR_MISALIGNED
    assert g(A, B, 0, 64, C, D, 0, 8, E, fw.BF16, 0) == fw.SUCCESS


def test_helpers_refuse_before_the_library():
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        fw.route(cpu, 2)
    with pytest.raises(ValueError):
        fw.route(cpu[0], 2)
    with pytest.raises(ValueError):
        fw.linear_int8(cpu.bfloat16(), cpu.to(torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        fw.linear_experts(cpu.bfloat16(), torch.zeros(2, 4, 8, dtype=torch.uint8), torch.zeros(2, 4),
                          torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        fw.combine(cpu.bfloat16(), torch.zeros(2, 2))
    with pytest.raises(ValueError):
        fw.quantize_experts(cpu)
    with pytest.raises(ValueError):
        fw.quantize_int8(cpu)
