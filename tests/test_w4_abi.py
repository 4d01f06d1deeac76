"""Argument checks of the 4-bit weight calls and of the few-token layer, without a GPU: invalid arguments are refused
before any HIP call (the pointers are never dereferenced)."""
import ctypes
import os

import pytest
import torch

import combine_router_gemm_amd as moe
from tests.test_abi import _layout

INVALID, UNSUPPORTED = -1, -2
P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.library_path()):
        pytest.skip("HIP library not built (python -m combine_router_gemm_amd.build)")
    return moe.load_library()


def test_sizes(lib):
    assert moe.moe_w4_codes_bytes(4096, 7168) == 4096 * 7168 // 2
    assert moe.moe_w4_scales_bytes(4096, 7168) == 4096 * 7168 // 32
    assert moe.moe_w4_codes_bytes(16, 32) == 1024 and moe.moe_w4_scales_bytes(16, 32) == 256
    assert moe.moe_w4_codes_bytes(16, 160) == 2048 and moe.moe_w4_scales_bytes(32, 544) == 1024
    for rows, K in ((8, 32), (16, 48), (0, 32), (16, 0), (-16, 32)):
        assert moe.moe_w4_codes_bytes(rows, K) == 0 and moe.moe_w4_scales_bytes(rows, K) == 0
    assert moe.moe_w4_shapes(3, 32, 160) == ((3, 2, 2, 1024), (3, 2, 1, 256))
    with pytest.raises(moe.MoeError):
        moe.moe_w4_shapes(8, 32)
    # beyond 32 bits
    assert moe.moe_w4_codes_bytes(1 << 24, 7168) == (1 << 24) * 3584
    assert moe.moe_layer_decode_workspace_bytes(0, 64, 8, 2, 32, moe.MOE_BF16) == 0
    assert moe.moe_layer_decode_workspace_bytes(33, 64, 8, 2, 32, moe.MOE_BF16) == 0
    assert moe.moe_layer_decode_workspace_bytes(32, 64, 8, 2, 32, moe.MOE_BF16) >= 64 * 32 * 4
    assert moe.moe_expert_mlp_w4_workspace_bytes(128, 8, 384, 8, 4, 2048) >= 1024 * 2048 * 2
    assert moe.moe_expert_mlp_w4_workspace_bytes(128, 8, 384, 7, 4, 2048) == 0


@pytest.mark.parametrize("name", ["moe_quantize_w4", "moe_dequantize_w4"])
def test_quantize_refusals(lib, name):
    def call(w=P, dt=moe.MOE_BF16, rows=32, K=64, c=P, s=P):
        if name == "moe_quantize_w4":
            return lib.moe_quantize_w4(w, dt, rows, K, c, s, None)
        return lib.moe_dequantize_w4(c, s, rows, K, w, dt, None)
    assert call(dt=5) == UNSUPPORTED
    assert call(rows=24) == UNSUPPORTED
    assert call(K=48) == UNSUPPORTED
    assert call(rows=-16) == INVALID
    assert call(K=0) == INVALID
    assert call(rows=1 << 60, K=64) == UNSUPPORTED
    for a in ("w", "c", "s"):
        assert call(**{a: None}) == INVALID
        assert call(**{a: ODD}) == INVALID
    assert call(rows=0, w=None, c=None, s=None) == 0


def test_expert_mlp_refusals(lib):
    def call(send=P, gc=P, gs=P, dc=P, ds=P, F=64, out=P, ws=P, wsb=1 << 40, **kw):
        kw.setdefault("H", 64)
        cl = _layout(**kw)
        return lib.moe_expert_mlp_w4(send, ctypes.byref(cl), gc, gs, dc, ds, F, out, ws, wsb, None)
    assert call(F=0) == INVALID
    assert call(F=48) == UNSUPPORTED
    assert call(H=72) == UNSUPPORTED
    assert call(H=60) == UNSUPPORTED
    assert call(wsb=16) == INVALID
    assert call(E=6, R=4) == INVALID
    assert call(k=9, E=16) == INVALID
    for a in ("send", "gc", "gs", "dc", "ds", "out", "ws"):
        assert call(**{a: None}) == INVALID
        assert call(**{a: ODD}) == INVALID
    # one expert's scales past 31 bits, though its rows are few
    assert call(F=1 << 28, T=1, k=1, E=1, R=1, C=1) == UNSUPPORTED
    assert call(F=1 << 27, T=1, k=1, E=1, R=1, C=1) == UNSUPPORTED
    assert call(F=1 << 26, H=1 << 13, T=1, k=1, E=1, R=1, C=1) == UNSUPPORTED
    assert lib.moe_expert_mlp_w4(P, None, P, P, P, P, 64, P, P, 1 << 40, None) == INVALID


@pytest.mark.parametrize("w4", [False, True])
def test_layer_refusals(lib, w4):
    def call(x=P, dt=moe.MOE_BF16, wr=P, bias=None, stride=0, T=4, H=64, E=8, R=1, k=2, C=4, F=64, gu=P, gs=P, dn=P,
             ds=P, lg=P, ids=P, w=P, y=P, ws=P, wsb=1 << 40):
        sizes = (T, H, E, R, k, C, F)
        if w4:
            return lib.moe_layer_decode_w4(x, wr, bias, stride, *sizes, gu, gs, dn, ds, lg, ids, w, y, ws, wsb, None)
        return lib.moe_layer_decode(x, dt, wr, bias, stride, *sizes, gu, dn, lg, ids, w, y, ws, wsb, None)
    if not w4:
        assert call(dt=7) == UNSUPPORTED
    assert call(T=33) == UNSUPPORTED
    assert call(T=-1) == INVALID
    assert call(E=513) == INVALID
    assert call(E=8, R=3) == INVALID
    assert call(R=0) == INVALID
    assert call(k=0) == INVALID
    assert call(k=9, E=16) == INVALID
    assert call(k=4, E=3) == INVALID
    assert call(C=-1) == INVALID
    assert call(F=0) == INVALID
    assert call(H=60) == UNSUPPORTED
    assert call(F=60) == UNSUPPORTED
    if w4:
        assert call(H=72) == UNSUPPORTED
        assert call(F=40) == UNSUPPORTED
    assert call(H=(1 << 23) + 32) == UNSUPPORTED
    assert call(F=(1 << 20) + 32) == UNSUPPORTED
    assert call(bias=P, stride=-1) == INVALID
    assert call(wsb=16) == INVALID
    names = ["x", "wr", "gu", "dn", "lg", "ids", "w", "y", "ws"] + (["gs", "ds"] if w4 else [])
    for a in names:
        assert call(**{a: None}) == INVALID
        assert call(**{a: ctypes.c_void_p(0x1002)}) == INVALID
    assert call(T=0, x=None, y=None, ws=None, wsb=0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    w = torch.zeros(32, 64)
    cs, ss = moe.moe_w4_shapes(32, 64)
    c, s = torch.zeros(cs, dtype=torch.uint8), torch.zeros(ss, dtype=torch.uint8)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_w4(w, c, s)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_w4(torch.zeros(24, 64), c, s)
    with pytest.raises(moe.MoeError):
        moe.moe_dequantize_w4(c, s, w)
