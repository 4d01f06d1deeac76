"""Argument checks of the router's training calls without a GPU, and their float64 references against autograd and against
differences."""
import ctypes
import os

import pytest
import torch

import combine_router_gemm_amd as moe
from tests._router_ref import balance, combine_backward, route_backward
from tests.test_abi import _layout

INVALID, UNSUPPORTED = -1, -2
P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.library_path()):
        pytest.skip("HIP library not built (python -m combine_router_gemm_amd.build)")
    return moe.load_library()


def test_balance_refusals(lib):
    def call(lg=P, ids=P, off=None, mask=None, T=4, E=8, k=2, S=1, w=1.0, loss=P, count=P, d=P, ws=P, wsb=1 << 40):
        return lib.moe_balance_loss(lg, ids, off, mask, T, E, k, S, w, loss, count, d, ws, wsb, None)
    assert call(T=-1) == INVALID
    assert call(E=0) == INVALID
    assert call(E=513) == INVALID
    assert call(k=0) == INVALID
    assert call(k=9, E=16) == INVALID
    assert call(k=4, E=3) == INVALID
    assert call(S=0, off=P) == INVALID
    assert call(S=2) == INVALID                      # several sequences need their offsets
    assert call(T=1 << 30, k=2) == UNSUPPORTED
    assert call(T=(1 << 30) + 1, k=1) == UNSUPPORTED
    assert call(S=1 << 30, off=P) == UNSUPPORTED
    assert call(wsb=16) == INVALID
    for a in ("lg", "ids", "loss", "count", "ws"):
        assert call(**{a: None}) == INVALID
    for a in ("lg", "ids", "off", "loss", "count", "d", "ws"):
        assert call(**{a: ODD}) == INVALID


def test_combine_backward_refusals(lib):
    def call(dy=P, dt=moe.MOE_BF16, out=P, w=P, dw=P, do=ctypes.c_void_p(0x2000), **kw):
        cl = _layout(**kw)
        return lib.moe_combine_backward(dy, dt, out, ctypes.byref(cl), w, dw, do, None)
    assert call(dt=4) == UNSUPPORTED
    assert call(H=60) == UNSUPPORTED
    assert call(E=6, R=4) == INVALID
    for a in ("dy", "out", "w", "dw"):
        assert call(**{a: None}) == INVALID
    for a in ("dy", "out", "w", "dw", "do"):
        assert call(**{a: ODD}) == INVALID
    assert call(do=P) == INVALID                     # not in place
    assert call(T=0, dy=None, out=None, w=None, dw=None, do=None) == 0
    assert lib.moe_combine_backward(P, moe.MOE_BF16, P, None, P, P, P, None) == INVALID


def test_route_backward_refusals(lib):
    def call(x=P, dt=moe.MOE_BF16, wr=P, ids=P, w=P, dw=P, di=P, T=4, H=64, E=8, k=2, dl=P, dx=P, dwr=P, db=P, ws=P,
             wsb=1 << 40):
        return lib.moe_route_backward(x, dt, wr, ids, w, dw, di, T, H, E, k, dl, dx, dwr, db, ws, wsb, None)
    assert call(dt=3) == UNSUPPORTED
    assert call(T=-1) == INVALID
    assert call(E=513) == INVALID
    assert call(k=9, E=16) == INVALID
    assert call(k=4, E=3) == INVALID
    assert call(H=0) == INVALID
    assert call(H=60) == UNSUPPORTED
    assert call(T=1 << 28, E=8) == UNSUPPORTED
    assert call(H=(1 << 21) + 8) == UNSUPPORTED
    assert call(dl=None) == INVALID
    assert call(dw=None, di=None) == INVALID         # no gradient at all
    assert call(ids=None) == INVALID
    assert call(w=None) == INVALID
    assert call(wr=None) == INVALID                  # d_x needs the weight
    assert call(x=None) == INVALID                   # d_w_router needs x
    for a in ("x", "wr", "ids", "w", "dw", "di", "dl", "dx", "dwr", "db", "ws"):
        assert call(**{a: ODD}) == INVALID
    if moe.moe_route_backward_workspace_bytes(4, 64, 8, moe.MOE_BF16):
        assert call(wsb=0) == INVALID


def test_workspace_sizes(lib):
    assert moe.moe_balance_loss_workspace_bytes(-1, 8, 1) == 0
    assert moe.moe_balance_loss_workspace_bytes(4, 0, 1) == 0
    assert moe.moe_balance_loss_workspace_bytes(4, 8, 0) == 0
    assert moe.moe_balance_loss_workspace_bytes(0, 8, 3) > 0
    assert moe.moe_balance_loss_workspace_bytes(1 << 20, 512, 4096) >= 4096 * 513 * 4
    assert moe.moe_route_backward_workspace_bytes(0, 64, 8, moe.MOE_BF16) == 0
    assert moe.moe_route_backward_workspace_bytes(4, 0, 8, moe.MOE_BF16) == 0


def test_reference_gradients_against_autograd_and_differences():
    g = torch.Generator().manual_seed(4)
    T, E, k, H = 9, 6, 2, 5
    logits = torch.randn(T, E, generator=g, dtype=torch.float64)
    ids = torch.argsort(logits, 1, descending=True)[:, :k]
    off, mask = [0, 4, 4, 8], torch.tensor([1, 1, 0, 1, 1, 1, 1, 1, 1])
    r = balance(logits, ids, 0.3, off, mask)
    eps = 1e-6
    for t, e in ((0, 0), (2, 1), (5, 3), (8, 2)):
        moved = []
        for sign in (1, -1):
            l2 = logits.clone()
            l2[t, e] += sign * eps
            moved.append(balance(l2, ids, 0.3, off, mask)["loss"])
        assert abs((moved[0] - moved[1]) / (2 * eps) - float(r["d"][t, e])) < 1e-9
    # the router: x -> logits -> softmax over the selected -> a function of the weights, and another of the logits
    x = torch.randn(T, H, generator=g, dtype=torch.float64).requires_grad_()
    wr = torch.randn(E, H, generator=g, dtype=torch.float64).requires_grad_()
    b = torch.randn(E, generator=g, dtype=torch.float64).requires_grad_()
    lg = x @ wr.T + b
    lg.retain_grad()
    sel = torch.argsort(lg.detach(), 1, descending=True)[:, :k]
    w = torch.softmax(torch.gather(lg, 1, sel), 1)
    cw, cl = torch.randn(T, k, generator=g, dtype=torch.float64), torch.randn(T, E, generator=g, dtype=torch.float64)
    ((w * cw).sum() + (lg * cl).sum()).backward()
    r = route_backward(x.detach(), wr.detach(), sel, w.detach(), cw, cl, False)
    for name, got in (("d_logits", lg.grad), ("d_x", x.grad), ("d_w_router", wr.grad), ("d_bias", b.grad)):
        assert torch.allclose(r[name][0], got, rtol=1e-12, atol=1e-13)
    # the combine
    out = torch.randn(7, H, generator=g, dtype=torch.float64).requires_grad_()
    row = torch.tensor([[0, 3], [-1, 1], [2, -1], [-1, -1], [6, 5]])
    w = torch.rand(5, 2, generator=g, dtype=torch.float64).requires_grad_()
    y = sum(torch.where(row[:, j:j + 1] >= 0, w[:, j:j + 1] * out[row[:, j].clamp(min=0)], torch.zeros(5, H).double())
            for j in range(2))
    dy = torch.randn(5, H, generator=g, dtype=torch.float64)
    y.backward(dy)
    d_w, _, d_out, _ = combine_backward(dy, out.detach(), row, w.detach())
    assert torch.allclose(d_w, w.grad, rtol=1e-12, atol=1e-13) and torch.allclose(d_out, out.grad, rtol=1e-12, atol=1e-13)


def test_binding_refuses_host_tensors(lib):
    lg, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(lg, ids, 1.0, torch.zeros(1), torch.zeros(1, 8, dtype=torch.int32))
    L = moe.Layout(4, 2, 4, 1, 4, 64, device="cpu")
    with pytest.raises(moe.MoeError):
        moe.moe_combine_backward(torch.zeros(4, 64), torch.zeros(8, 64), L, torch.zeros(4, 2), torch.zeros(4, 2))
    with pytest.raises(moe.MoeError):
        moe.moe_route_backward(torch.zeros(4, 64), torch.zeros(8, 64), ids, torch.zeros(4, 2), torch.zeros(4, 2), None, lg)


def test_route_backward_more_refusals(lib):
    at = lambda a: ctypes.c_void_p(a)

    def call(x=P, dx=at(0x2000), dwr=at(0x4000), T=4, H=64, E=8):
        return lib.moe_route_backward(x, moe.MOE_BF16, P, P, P, P, P, T, H, E, 1, P, dx, dwr, None, P, 0, None)
    assert call() == INVALID                          # the workspace is too small, and nothing else
    assert call(T=(1 << 26) + 1, H=8, E=1) == UNSUPPORTED
    # a workspace that suffices: only the aliases are left to refuse
    def full(x, dx, dwr):
        return lib.moe_route_backward(x, moe.MOE_BF16, P, P, P, P, P, 4, 64, 8, 1, P, dx, dwr, None, P, 1 << 40, None)
    assert full(P, P, at(0x4000)) == INVALID          # d_x in place of x, which d_w_router reads
    assert full(P, at(0x2000), at(0x2000)) == INVALID
