"""Every tile height of the 4-bit expert MLP, with the height that a case takes asserted: sizes for 256 compute units, one
and two ranks, K not a multiple of a stage's 64, a last column tile that is partly empty, ragged and empty experts."""
import ctypes

import pytest
import torch

import combine_router_gemm_amd as moe
from tests._layer_ref import expert, within
from tests.test_gpu_w4 import DEV, case

# name, counts, T, k, R, C, H, F, rows per tile, parts of the down pass
CASES = [
    ("t32", [33, 0, 16, 70, 1, 5], 130, 1, 1, 70, 160, 96, 32, 1),
    ("t32_ranks", [17, 64, 0, 31, 2, 40, 33, 1], 100, 2, 2, 64, 288, 352, 32, 1),
    ("t32_one_set", [5, 0, 40, 3, 33, 1], 90, 1, 6, 40, 96, 160, 32, 1),  # every rank's rows share one weight set
    ("t32_split", [9, 0, 32, 1], 42, 1, 1, 42, 160, 2304, 32, 2),
    ("t32_split_ranks", [3, 16, 0, 1, 7, 20], 47, 1, 2, 20, 64, 4160, 32, 3),
    ("t128", [640, 129, 0, 1, 257, 500, 64, 33], 5120, 2, 1, 5120, 288, 2016, 128, 1),
    ("t128_ranks", [512, 1, 0, 300, 255, 17, 128, 33, 256, 0, 31, 90, 1, 400, 64, 129], 5120, 2, 2, 1024, 288, 2016,
     128, 1),
    ("t256", [2049, 255, 0, 1400], 8192, 1, 1, 8192, 1056, 544, 256, 1),
    ("t256_ranks", [511, 1, 0, 300, 700, 256, 33, 1025], 4096, 2, 2, 2048, 1056, 544, 256, 1),
]
IDS = [c[0] for c in CASES]


@pytest.mark.parametrize("name,counts,T,k,R,C,H,F,tile,parts", CASES, ids=IDS)
def test_cases_take_the_tiles_they_are_meant_for(name, counts, T, k, R, C, H, F, tile, parts):
    assert moe.moe_expert_mlp_w4_tiling(T, k, len(counts), R, C, H, F) == (tile, parts)


def test_tiling_refuses_what_the_call_refuses():
    lib = moe.load_library()

    def call(T=8, k=2, E=8, R=1, C=8, H=64, F=64):
        rows, parts = ctypes.c_int(-5), ctypes.c_int(-5)
        st = lib.moe_expert_mlp_w4_tiling(T, k, E, R, C, H, F, ctypes.byref(rows), ctypes.byref(parts))
        assert st == 0 or (rows.value, parts.value) == (-5, -5)
        return st
    assert call() == 0 and call(T=0) == 0 and call(C=0) == 0
    for bad in (dict(T=-1), dict(C=-1), dict(E=0), dict(E=513), dict(R=3), dict(R=0), dict(k=0), dict(k=9, E=16),
                dict(k=4, E=3), dict(H=0), dict(F=0)):
        assert call(**bad) == -1, bad
    for bad in (dict(H=48), dict(F=40), dict(F=1 << 28, T=1, k=1, E=1, C=1), dict(T=1 << 20, C=1 << 20, F=1 << 12),
                dict(T=1 << 30, k=8)):
        assert call(**bad) == -2, bad
    one = ctypes.byref(ctypes.c_int())
    assert lib.moe_expert_mlp_w4_tiling(8, 2, 8, 1, 8, 64, 64, None, one) == -1
    assert lib.moe_expert_mlp_w4_tiling(8, 2, 8, 1, 8, 64, 64, one, None) == -1
    with pytest.raises(moe.MoeError):
        moe.moe_expert_mlp_w4_tiling(8, 2, 8, 1, 8, 48, 64)


def some_rows(counts, step):
    """(expert, rows): every `step`-th row, the rows at the borders of 32-row blocks near 128 and 256, the last one."""
    at = 0
    for e, n in enumerate(counts):
        rows = set(range(0, n, step)) | {r for r in (15, 16, 31, 32, 127, 128, 255, 256, 511, 512, n - 1) if 0 <= r < n}
        if rows:
            yield e, [at + r for r in sorted(rows)]
        at += n


def run(counts, T, k, R, C, H, F, L, send, packs):
    """The output, with rows past the last kept one checked; a second call on another workspace is bit-identical."""
    n = moe.moe_expert_mlp_w4_workspace_bytes(T, k, len(counts), R, C, F)
    outs = []
    for fill in (0xFF, 0x11):
        out = torch.full((L.rows_max, H), -7.0, dtype=torch.bfloat16, device=DEV)
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out, workspace=ws)
        assert torch.all(out[sum(counts):] == -7.0)
        outs.append(out)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    return outs[0]


@pytest.mark.gpu
@pytest.mark.parametrize("name,counts,T,k,R,C,H,F,tile,parts", CASES, ids=IDS)
def test_every_tile_height(name, counts, T, k, R, C, H, F, tile, parts):
    print(f"\n[gpu] expert MLP w4 tiles {name}", flush=True)
    assert moe.moe_expert_mlp_w4_tiling(T, k, len(counts), R, C, H, F) == (tile, parts)
    L, send, packs, vals = case(counts, T, k, R, C, H, F, 300 + len(name))
    out = run(counts, T, k, R, C, H, F, L, send, packs).cpu()
    El = len(counts) // R
    half = 2.0 ** -16 if tile == 32 else 2.0 ** -8  # of h: two bf16 parts or one
    for e, rows in some_rows(counts, 1 if sum(counts) < 300 else 7):
        ref, b = expert(send[rows].double(), vals[0][e % El], vals[1][e % El], half)
        assert within(out[rows], ref, b, torch.bfloat16) <= 1.0, e
