"""GPU: infinities in the down weights and sums beyond float32 in the calls that keep h in two bf16 parts. The formula's
result is an infinity; the second part's product (0 * inf, or an infinity of the other sign) must not make it NaN."""
import pytest
import torch

import combine_router_gemm_amd as moe
from tests.test_gpu_decode import DEV, Run, inputs, pack4
from tests.test_gpu_w4 import layout_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,F,H", [(1, 1, 32, 32), (3, 2, 72, 40), (20, 2, 64, 64), (32, 1, 1056, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_an_infinite_down_weight_gives_an_infinity(T, k, F, H, dtype):
    """k = F - 3 of h is positive everywhere, and n = 5 of every expert's down weight is infinite there: y[:, 5] is
    +inf, y[:, 6] with the opposite sign -inf, whatever the remainder of h is (none for h = 2, either sign else)."""
    E = 4
    inp = inputs("inf_down", T, H, E, k, F, 1, dtype, "uniform", 30 + T)
    x, gu, dn = inp["x"], inp["w_gate_up"], inp["w_down"]
    x[:, 0] = 1.0
    gu[:, F - 3], gu[:, 2 * F - 3] = 0.0, 0.0
    # silu(g) = g for g = 64 in float32; h = 64 u
    gu[:, F - 3, 0] = 64.0
    for e, u in enumerate((2.0 ** -5, 1.0 + 2.0 ** -7, 1.5, 1.0)):
        gu[e, 2 * F - 3, 0] = u
        gu[e, 2 * F - 3, 1] = (0.0, 0.0, 2.0 ** -7, -(2.0 ** -7))[e]
    x[:, 1] = torch.where(torch.arange(T, device=DEV) % 2 == 0, 0.25, 0.375).to(dtype)
    clean = Run(inp, k, 1, T)().outputs()
    dn[:, 5, F - 3], dn[:, 6, F - 3] = float("inf"), float("-inf")
    y = Run(inp, k, 1, T)().outputs()[3]
    assert torch.all(y[:, 5] == float("inf")) and torch.all(y[:, 6] == float("-inf"))
    rest = [n for n in range(H) if n not in (5, 6)]
    assert torch.equal(y[:, rest], clean[3][:, rest])


def large_h(El, H, F):
    """Weights whose h_3 is 2^120 - 2^111 for x = 1 (the nearest bf16 is 2^120, the remainder negative) and whose down
    weight there is 2^125: the product is beyond float32, and so is the remainder's, with the other sign."""
    gu = torch.zeros(El, 2 * F, H, dtype=torch.bfloat16, device=DEV)
    gu[:, 3, 0] = 2.0 ** 60
    gu[:, F + 3, 0], gu[:, F + 3, 32] = 2.0 ** 60, -(2.0 ** 51)
    dn = torch.zeros(El, H, F, dtype=torch.bfloat16, device=DEV)
    dn[:, :, 3] = 2.0 ** 125
    return gu, dn


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("T", [1, 7, 20])
def test_a_layer_beyond_float32_is_an_infinity(T, w4):
    H, F = 64, 32
    inp = inputs("big", T, H, 1, 1, F, 1, torch.bfloat16, "uniform", 8)
    inp["x"].fill_(1.0)
    inp["w_gate_up"], inp["w_down"] = large_h(1, H, F)
    packs = pack4(inp["w_gate_up"])[0] + pack4(inp["w_down"])[0] if w4 else None
    assert torch.all(Run(inp, 1, 1, T, packs)().y == float("inf"))


def test_rows_beyond_float32_are_not_finite():
    """moe_expert_mlp_w4 adds both parts of h in one sum for experts of more than 16 rows: an infinity or NaN there, an
    infinity for up to 16 rows."""
    counts, H, F = [2, 20, 16], 64, 32
    L = layout_of(counts, 38, 1, 1, 38, H)
    assert moe.moe_expert_mlp_w4_tiling(38, 1, 3, 1, 38, H, F)[0] == 32
    packs = [t for w in large_h(3, H, F) for t in pack4(w)[0]]
    out = torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_mlp_w4(torch.ones(L.rows_max, H, dtype=torch.bfloat16, device=DEV), L, *packs, out)
    assert torch.all(out[:2] == float("inf")) and torch.all(out[22:38] == float("inf"))
    assert not torch.isfinite(out[2:22].float()).any()
