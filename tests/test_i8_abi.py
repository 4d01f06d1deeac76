"""Argument checks of the int8 calls without a GPU (invalid arguments are refused before any HIP call; the pointers are
never dereferenced), and the float64 reference against whole-number arithmetic."""
import ctypes
import os
import random

import pytest
import torch

import combine_router_gemm_amd as moe
from tests._i8_ref import level_by_fractions, levels
from tests.test_abi import _layout

INVALID, UNSUPPORTED = -1, -2
P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.library_path()):
        pytest.skip("HIP library not built (python -m combine_router_gemm_amd.build)")
    return moe.load_library()


def test_reference_levels():
    rng = random.Random(3)
    rows = [[127.0, 63.5, -0.5, 0.5, 1.5, -2.5, 0.0, -127.0],      # every quotient a whole number or a tie
            [1.0, 0.5, 0.25, -0.125, 1.0 / 128, -0.0, 3.0 / 254, 0.75],
            [2.0 ** -149, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, -2.0 ** -149],
            [2.0 ** 127, 2.0 ** 126, 2.0 ** 119, -2.0 ** 120, 1.0, 2.0 ** -149, 0.0, 0.0]]
    rows += [[float(torch.tensor(rng.gauss(0, 1)).bfloat16()) for _ in range(8)] for _ in range(50)]
    v = torch.tensor(rows).double()  # float32 values, as levels takes them
    lv, top = levels(v)
    for r, row in enumerate(v.tolist()):
        assert [int(x) for x in lv[r]] == [level_by_fractions(x, float(top[r])) for x in row]


@pytest.mark.parametrize("name", ["moe_quantize_i8", "moe_dequantize_i8"])
def test_quantize_refusals(lib, name):
    def call(w=P, dt=moe.MOE_BF16, rows=31, K=64, c=P, s=P):
        if name == "moe_quantize_i8":
            return lib.moe_quantize_i8(w, dt, rows, K, c, s, None)
        return lib.moe_dequantize_i8(c, s, rows, K, w, dt, None)
    assert call(dt=5) == UNSUPPORTED
    assert call(K=40) == UNSUPPORTED
    assert call(rows=-1) == INVALID
    assert call(K=0) == INVALID
    assert call(rows=1 << 60, K=64) == UNSUPPORTED
    for a in ("w", "c", "s"):
        assert call(**{a: None}) == INVALID
        assert call(**{a: ODD}) == INVALID
    assert call(rows=0, w=None, c=None, s=None) == 0


def test_dispatch_refusals(lib):
    def call(x=P, dt=moe.MOE_BF16, ids=P, q=P, s=P, ws=P, wsb=1 << 40, **kw):
        kw.setdefault("H", 64)
        cl = _layout(**kw)
        return lib.moe_dispatch_i8(x, dt, ids, ctypes.byref(cl), q, s, ws, wsb, None)
    assert call(dt=moe.MOE_F32) == UNSUPPORTED
    assert call(H=72) == UNSUPPORTED
    assert call(H=60) == UNSUPPORTED
    assert call(wsb=16) == INVALID
    assert call(E=6, R=4) == INVALID
    for a in ("x", "ids", "q", "s", "ws"):
        assert call(**{a: None}) == INVALID
        assert call(**{a: ODD}) == INVALID
    assert lib.moe_dispatch_i8(P, moe.MOE_BF16, P, None, P, P, P, 1 << 40, None) == INVALID


def test_expert_mlp_refusals(lib):
    def call(q=P, s=P, gc=P, gs=P, dc=P, ds=P, F=64, out=P, ws=P, wsb=1 << 40, **kw):
        kw.setdefault("H", 64)
        cl = _layout(**kw)
        return lib.moe_expert_mlp_i8(q, s, ctypes.byref(cl), gc, gs, dc, ds, F, out, ws, wsb, None)
    assert call(F=0) == INVALID
    assert call(F=-16) == INVALID
    assert call(F=40) == UNSUPPORTED
    assert call(H=72) == UNSUPPORTED
    assert call(wsb=16) == INVALID
    assert call(k=9, E=16) == INVALID
    for a in ("q", "s", "gc", "gs", "dc", "ds", "out", "ws"):
        assert call(**{a: None}) == INVALID
        assert call(**{a: ODD}) == INVALID
    one = dict(T=1, k=1, E=1, R=1, C=1)
    assert call(F=1 << 17, **one) == UNSUPPORTED           # an int32 sum could overflow
    assert call(H=1 << 17, **one) == UNSUPPORTED
    assert call(F=1 << 16, H=1 << 14, **one) == UNSUPPORTED  # an expert's weights past 31 bits
    assert call(T=1 << 20, k=1, E=1, R=1, C=1 << 20, H=4096) == UNSUPPORTED  # rows past 31 bits
    assert lib.moe_expert_mlp_i8(P, P, None, P, P, P, P, 64, P, P, 1 << 40, None) == INVALID


def test_workspace_sizes(lib):
    size = moe.moe_expert_mlp_i8_workspace_bytes
    rows = moe.moe_rows_max(128, 8, 384, 4)
    assert size(128, 8, 384, 8, 4, 7168, 2048) >= rows * 2048 * 5
    assert size(128, 8, 384, 7, 4, 7168, 2048) == 0
    assert size(1, 1, 1, 1, 1, 1 << 17, 64) == 0
    assert size(1, 1, 1, 1, 1, 0, 64) == 0
    # beyond 32 bits
    assert size(1 << 20, 1, 1, 1, 1 << 20, 64, 2032) >= (1 << 20) * 2032 * 5


def test_tiling_query(lib):
    """Every tile, and each split, is what some sizes take (tests/test_gpu_i8.py has the same sizes on the GPU)."""
    from tests.test_gpu_i8 import CASES
    seen = set()
    for name, counts, T, k, R, C, H, F, rows, gu, dn in CASES:
        t = moe.moe_expert_mlp_i8_tiling(T, k, len(counts), R, C, H, F)
        assert (t[0], t[1] > 1, t[2] > 1) == (rows, gu, dn), (name, t)
        seen.add(rows)
    assert seen == {32, 64, 128, 256}
    n = [ctypes.c_int(7) for _ in range(3)]
    call = lambda T=4, k=2, E=8, R=1, C=4, H=64, F=64, out=n: lib.moe_expert_mlp_i8_tiling(
        T, k, E, R, C, H, F, *[ctypes.byref(v) if v is not None else None for v in out])
    assert call(H=72) == UNSUPPORTED and call(F=0) == INVALID and call(k=9, E=16) == INVALID and call(R=3) == INVALID
    assert call(T=-1) == INVALID and call(out=[n[0], None, n[1]]) == INVALID and call(F=1 << 17) == UNSUPPORTED
    assert [v.value for v in n] == [7, 7, 7]
    assert call() == 0 and [v.value for v in n] != [7, 7, 7]


def test_binding_refuses_host_tensors(lib):
    w, q, s = torch.zeros(32, 64), torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_i8(w, q, s)
    with pytest.raises(moe.MoeError):
        moe.moe_dequantize_i8(q, s, w)
    L = moe.Layout(4, 2, 4, 1, 4, 64, device="cpu")
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch_i8(torch.zeros(4, 64, dtype=torch.bfloat16), ids, L, torch.zeros(8, 64, dtype=torch.int8),
                            torch.zeros(8))
    with pytest.raises(moe.MoeError):
        moe.moe_expert_mlp_i8(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8), L,
                              torch.zeros(4, 64, 64, dtype=torch.int8), torch.zeros(4, 64),
                              torch.zeros(4, 64, 32, dtype=torch.int8), torch.zeros(4, 64),
                              torch.zeros(8, 64, dtype=torch.bfloat16))
