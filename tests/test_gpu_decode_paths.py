"""GPU: paths of the 4-bit few-token layer that ordinary widths do not take, on the sparse weights of
tests/test_sparse_experts.py: runs of K longer than the scale tiles that LDS holds at a time (more than 16 steps of 128 per
wave, in gate/up and in the down pass), and four waves to a gate/up tile. The counts in the comments are for 256 CUs."""
import pytest
import torch

import tests._layer_ref as ref
import tests.test_sparse_experts as sparse
from tests._layer_ref import layer, within
from tests.test_gpu_decode import DEV, Run, pack4
from tests.test_sparse_experts import expert, rows_of, weights

pytestmark = pytest.mark.gpu


def check(monkeypatch, T, H, El, k, F, seed):
    """Token t chooses experts t k .. t k + k - 1 (mod El). All experts share one packed weight set, odd ones with the
    signs of the down weights flipped."""
    gu, dn = weights(1, F, H)
    packs = []
    for i, w in enumerate((gu, dn)):
        (c, s), _ = pack4(w.to(DEV))
        c = c.repeat(El, 1, 1, 1)
        if i == 1:
            c[1::2] ^= 0x88
        packs += [c, s.repeat(El, 1, 1, 1)]
    gu, dn = gu[0].double(), dn[0].double()
    bias = torch.randn(T, El, generator=torch.Generator().manual_seed(seed))
    for t in range(T):
        bias[t, [(t * k + j) % El for j in range(k)]] += 100.0
    inp = {"x": rows_of(T, H, seed + 1).to(DEV), "w_router": torch.zeros(El, H, device=DEV), "bias": bias.to(DEV),
           "w_down": torch.empty(0, H, F)}
    r = Run(inp, k, 1, T, packs)()
    again = Run(inp, k, 1, T, packs)()
    torch.cuda.synchronize()
    assert torch.equal(r.y.view(torch.int16), again.y.view(torch.int16))
    ids = r.ids.cpu().long()
    for t in range(T):
        assert sorted(ids[t].tolist()) == sorted((t * k + j) % El for j in range(k))
    monkeypatch.setattr(ref, "expert", expert)
    want = layer(inp["x"].cpu().double(), torch.zeros(El, H, dtype=torch.float64), bias.double(), k, 1, T, ids,
                 lambda l: (gu, -dn if l % 2 else dn), 2.0 ** -16)
    assert within(r.y.cpu(), want["y"], want["dy"], torch.bfloat16) <= 1.0


# 130 and 261 steps of K, 17 and 33 per wave; up to 4, up to 16 and more rows of an expert; H past a scale tile by 160
# and by 96
@pytest.mark.parametrize("H", [16544, 33376])
@pytest.mark.parametrize("T,El", [(3, 2), (9, 1), (20, 1)])
def test_gate_up_over_several_chunks_of_scales(monkeypatch, T, El, H):
    print(f"\n[gpu] layer w4 chunks T {T} experts {El} H {H}", flush=True)
    check(monkeypatch, T, H, El, 1, 32, 700 + T)


# 2049 steps of K (two experts: 4098) in 128 runs of 17 (33): eight parts of sixteen waves
@pytest.mark.parametrize("T,El", [(1, 1), (2, 2), (12, 1)])
def test_down_over_several_chunks_of_scales(monkeypatch, T, El):
    print(f"\n[gpu] layer w4 long F T {T} experts {El}", flush=True)
    check(monkeypatch, T, 64, El, 1, 262176, 720 + T)


# tiles of 32 columns over all experts: 40 x 32 = 1280, fewer than the 2048 that two waves each would need; and
# 32 x 64 = 2048 with 29 steps, too few for eight waves and too many for two
@pytest.mark.parametrize("T,El,k,F,H", [(24, 40, 4, 1024, 96), (10, 40, 4, 1024, 544), (8, 32, 4, 2048, 3680)])
def test_four_waves_to_a_gate_up_tile(monkeypatch, T, El, k, F, H):
    print(f"\n[gpu] layer w4 four waves T {T} experts {El} H {H} F {F}", flush=True)
    check(monkeypatch, T, H, El, k, F, 740 + T)


# every (token, slot) pair chooses an expert of its own: 256 rows and as many experts, the most a call can have
@pytest.mark.parametrize("El", [256, 512])
def test_as_many_experts_as_pairs(monkeypatch, El):
    print(f"\n[gpu] layer w4 256 rows of 256 experts of {El}", flush=True)
    check(monkeypatch, 32, 96, El, 8, 64, 760)


# R == E: one weight set, so a token's kept choices are one row with the sum of their weights; with a capacity and without
@pytest.mark.parametrize("kind", ["f32", "bf16", "w4"])
@pytest.mark.parametrize("T,C", [(1, 1), (7, 2), (32, 32)])
def test_one_weight_set_for_every_expert(monkeypatch, T, C, kind):
    sparse.test_layer(monkeypatch, "one_set", T, 96, 8, 8, 64, 8, C, "uniform", kind)
