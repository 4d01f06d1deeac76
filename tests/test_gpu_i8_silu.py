"""GPU: silu of the int8 expert MLP at the ends of float32's range, read out code by code.

Every gate of a row has the same g (one non-zero code), and the up half gives whole levels, of which one is 127: h = silu(g) u
has the levels as its codes whatever silu is, as long as it is neither 0 nor NaN, and the down weights pick one of them for each
output. What is off: g by two float32 roundings, so silu by |g| 2^-23 of itself where it falls exponentially, SILU_REL, and, where
silu is subnormal in float32, one step of 2^-149; the scale, its product and the bf16 rounding are counted by `within`."""
import pytest
import torch

import combine_router_gemm_amd as moe
from tests._layer_ref import SILU_REL, U, within
from tests.test_gpu_w4 import layout_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HUGE = [3.0e38, 2.4e38, 2.3e38, 1.0e38, 1.0e30, 2.0e5]
LOW = [-0.5, -30.0, -63.0, -64.5, -80.0, -87.0, -87.4, -88.0, -88.7, -88.8, -90.0, -95.0, -100.0, -102.0]
GONE = [-200.0, -1.0e9, -3.0e38]  # silu below half of float32's smallest step


# H, F, rows per tile, whether the gate/up pass is split
@pytest.mark.parametrize("H,F,copies,tile,split", [(16, 32, 1, 32, False), (2064, 48, 1, 32, True), (32, 32, 40, 32, False),
                                                        (512, 512, 100, 64, False), (512, 512, 300, 128, False),
                                                        (1184, 736, 300, 256, False)])
def test_ends_of_silu(H, F, copies, tile, split):
    print(f"\n[gpu] silu of int8 experts {H} {F} {copies}", flush=True)
    g = torch.Generator().manual_seed(H)
    goal = [HUGE * copies, LOW * copies, GONE * copies]
    counts = [len(v) for v in goal]
    T = sum(counts)
    cut = moe.moe_expert_mlp_i8_tiling(T, 1, 3, 1, T, H, F)
    assert (cut[0], cut[1] > 1) == (tile, split)
    L = layout_of(counts, T, 1, 1, T, H)
    levels = torch.randint(-127, 128, (3, F), generator=g)
    levels[:, 0] = 127
    gu, dn = torch.zeros(3, 2 * F, H, dtype=torch.int8), torch.zeros(3, H, F, dtype=torch.int8)
    gu[:, :F, 0] = 1
    gu[:, F:, 1] = levels.to(torch.int8)
    n = min(H, F)
    dn[:, torch.arange(n), torch.arange(n)] = 1
    gu_s, dn_s = torch.empty(3, 2 * F), torch.ones(3, H)
    gu_s[0, :F], gu_s[0, F:] = 2.0 ** 40, 2.0 ** -90  # u is at most 0.25 where g is 3e38
    gu_s[1, :F], gu_s[1, F:] = 1.0, 2.0 ** 20         # and large where silu is tiny
    gu_s[2, :F], gu_s[2, F:] = 1.0, 2.0 ** -90
    g_goal = torch.tensor(sum(goal, []), dtype=torch.float64)
    expert = torch.repeat_interleave(torch.arange(3), torch.tensor(counts))
    q = torch.zeros(L.rows_max, H, dtype=torch.int8)
    q[:T, 0] = torch.where(g_goal < 0, -127, 127).to(torch.int8)
    q[:T, 1] = 1
    s = torch.zeros(L.rows_max)
    s[:T] = (g_goal.abs() / (127.0 * gu_s[expert, 0].double())).float()
    out = torch.full((L.rows_max, H), -7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_mlp_i8(q.to(DEV), s.to(DEV), L, gu.to(DEV), gu_s.to(DEV), dn.to(DEV), dn_s.to(DEV), out)
    s64 = s[:T].double()
    gate = q[:T, 0].double() * s64 * gu_s[expert, 0].double()
    unit = s64 * gu_s[expert, F].double()
    # silu(g) = g e^g / (1 + e^g) below 0, without an overflow
    e = torch.exp(-gate.abs())
    silu = torch.where(gate < 0, gate * e / (1.0 + e), gate / (1.0 + e))
    ref = torch.zeros(T, H, dtype=torch.float64)
    ref[:, :n] = silu.unsqueeze(1) * unit.unsqueeze(1) * levels[expert, :n].double()
    big = unit.unsqueeze(1) * levels[expert, :n].double().abs()
    bound = torch.zeros_like(ref)
    rel = torch.where(gate < 0, gate.abs() * 3 * U, torch.full_like(gate, 3 * U)) + SILU_REL + 8 * U
    bound[:, :n] = (rel * silu.abs() + 2.0 ** -149).unsqueeze(1) * big
    gone = gate < -104.0
    got = out[:T].cpu()
    assert not got[gone].any()  # (zeros of either sign)
    assert within(got[~gone], ref[~gone], bound[~gone], torch.bfloat16) <= 1.0
