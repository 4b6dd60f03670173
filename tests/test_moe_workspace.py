"""Workspaces of the mixture-of-experts and int8 calls: the products grouped by
expert need none and take no notice of one, the router's and the int8 layer's are
checked. No call here reaches a kernel launch but the one marked for the GPU."""
import types

import pytest
import torch

import fp8_weight_only_amd as fw
from test_moe_abi import A, E, F, G, H, I, _experts, _int8, _route

SIZES = [(1, 4, 256, 8192), (8, 64, 512, 4096), (2, 8, 1024, 14336), (1, 8, 14336, 4096), (512, 128, 4096, 1024),
         (1332, 60, 1030, 1001), (8192, 8, 14336, 4096), (100000, 8, 512, 256)]


@pytest.mark.parametrize("m,e,n,k", SIZES)
def test_experts_need_no_workspace(m, e, n, k):
    for x, q in ((0, 0), (A, E), (A + 2, E + 1)):
        assert fw.fp8w_linear_experts_workspace_bytes(m, e, n, k, x, q) == 0


@pytest.mark.parametrize("ws,wsb", [(0, 0), (0, 1 << 20), (I, 0), (I, 1 << 20), (I + 1, 7), (A, 1 << 20), (H, 1 << 20)])
def test_experts_take_no_notice_of_a_workspace(ws, wsb):
    """NULL, short, misaligned or inside another buffer: neither refused nor used."""
    assert _experts(m=0, xc=0, xr=0, ws=ws, wsb=wsb) == fw.SUCCESS
    assert _experts(n=0, ws=ws, wsb=wsb) == fw.SUCCESS
    assert _experts(y=A, ws=ws, wsb=wsb) == fw.ERR_INVALID_VALUE  # the other checks stand


def test_experts_helper_runs_the_same_way_with_a_workspace(monkeypatch):
    calls = []
    monkeypatch.setattr(fw.moe, "_FAST", types.SimpleNamespace(linear_experts=lambda *a: calls.append(a) or "made"))
    t = torch.zeros(4, 8)
    assert fw.linear_experts(t, t, t, t) == "made"
    assert fw.linear_experts(t, t, t, t, workspace=torch.empty(64, dtype=torch.uint8)) == "made"
    assert len(calls) == 2 and calls[0] == calls[1]


def test_route_workspace_is_checked():
    """Two launches need one; its absence, shortness, misalignment and overlap are refused."""
    need = fw.fp8w_route_workspace_bytes(100000, 64, 2)
    assert need > 0
    big = dict(t=100000, e=64)
    assert _route(wsb=need - 1, **big) == fw.ERR_WORKSPACE
    assert _route(ws=0, wsb=need, **big) == fw.ERR_WORKSPACE
    assert _route(ws=G + 2, wsb=need, **big) == fw.ERR_MISALIGNED
    for other in (A, E, F, F + 4 * 2 * 100000 - 4):
        assert _route(ws=other, wsb=need, **big) == fw.ERR_INVALID_VALUE
    assert fw.fp8w_route_workspace_bytes(1, 64, 2) == 0


@pytest.mark.parametrize("m,n,k", [(22, 4096, 14336), (4096, 128, 256), (130, 512, 8192), (70, 300, 8198)])
def test_int8_workspace_is_checked(m, n, k):
    need = fw.fp8w_linear_int8_workspace_bytes(m, n, k, A, E)
    assert need > 0
    size = dict(m=m, n=n, k=k, q=E, y=H)
    assert _int8(wsb=need - 1, **size) == fw.ERR_WORKSPACE
    assert _int8(ws=0, wsb=need, **size) == fw.ERR_WORKSPACE
    assert _int8(ws=F + 8, wsb=need, **size) == fw.ERR_MISALIGNED
    for other in (A, E, H):
        assert _int8(ws=other, wsb=need, **size) == fw.ERR_INVALID_VALUE


@pytest.mark.gpu
def test_experts_with_a_workspace_give_the_same_bits():
    g = torch.Generator(device="cuda").manual_seed(0)
    q, s = fw.quantize_experts(torch.randn((8, 512, 1024), generator=g, device="cuda"))
    x = torch.randn((40, 1024), generator=g, device="cuda").bfloat16()
    offsets = torch.arange(0, 45, 5, device="cuda").int()
    want = fw.linear_experts(x, q, s, offsets)
    ws = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    assert torch.equal(fw.linear_experts(x, q, s, offsets, workspace=ws), want) and (ws == 7).all()
