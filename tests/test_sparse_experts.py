"""The expert products on weights with a few non-zeros per row, where the bounds are tight: every k of every product
reaches some output, and h that lost its second part, or has it from another row, is outside its bound.

Adding a product that is exactly zero rounds nothing, so a sum of n products with m non-zero ones is off by at most
(m + 1) 2^-24 times the sum of their absolute values; the other terms are those of tests/_layer_ref.py. The CPU tests
plant the mistakes in a float64 form of the kernels and ask that the bound rejects each of them."""
import pytest
import torch

import combine_router_gemm_amd as moe
import tests._layer_ref as ref
from tests._layer_ref import SILU_REL, U, layer, within
from tests.test_gpu_decode import CASES as LAYER_CASES
from tests.test_gpu_decode import DEV, Run, pack4
from tests.test_gpu_w4 import layout_of
from tests.test_w4_tiles import CASES, IDS, run, some_rows


def sparse(El, N, K, shift):
    """[El, N, K]: rows of two non-zeros, or of two per N columns where K > N; every column has some. The values are
    4-bit codes at one scale, so quantising them changes nothing."""
    P = min(N, K)
    n, k = torch.arange(N)[:, None], torch.arange(K)[None, :]
    a = ((k - n - shift) % P == 0).double() * torch.where((n // P) % 2 == 0, 1.5, 0.75)
    b = ((k - 2 * n - shift - 1) % P == 0).double() * torch.where(n % 2 == 0, 1.0, -0.5)
    sign = torch.where(torch.arange(El) % 2 == 0, 1.0, -1.0)[:, None, None].double()
    w = torch.where(a != 0, a, -b) * sign
    assert ((w != 0).any(0) if El == 1 else (w[0] != 0)).any(0).all()
    return w.to(torch.bfloat16)


def weights(El, F, H):
    return torch.cat([sparse(El, F, H, 0), sparse(El, F, H, 7)], 1), sparse(El, H, F, 3)


def expert(rows, gate_up, down, h_half_step):
    """tests/_layer_ref.py's expert with the bounds of sums of few non-zero products."""
    F = down.shape[1]
    m1 = int((gate_up != 0).sum(1).max()) + 1
    m2 = int((down != 0).sum(1).max()) + 1
    s = rows @ gate_up.T
    ds = m1 * U * (rows.abs() @ gate_up.abs().T)
    g, u, dg, du = s[:, :F], s[:, F:], ds[:, :F], ds[:, F:]
    act = g / (1.0 + torch.exp(-g))
    h = act * u
    dh = (1.1 * dg + SILU_REL * act.abs()) * (u.abs() + du) + act.abs() * du
    dh = dh + h_half_step * (h.abs() + dh)
    out = h @ down.T
    return out, dh @ down.abs().T + m2 * U * ((h.abs() + dh) @ down.abs().T)


def rows_of(n, H, seed):
    return torch.randn(n, H, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


MISTAKES = {
    "none": lambda hi, lo: hi + lo,
    "second part lost": lambda hi, lo: hi,
    "second part subtracted": lambda hi, lo: hi - lo,
    "second part of another row": lambda hi, lo: hi + lo.roll(1, 0),
    "second part of another column": lambda hi, lo: hi + lo.roll(1, 1),
    "a column lost": lambda hi, lo: (hi + lo) * (torch.arange(hi.shape[1]) != hi.shape[1] - 2),
    "last step's columns lost": lambda hi, lo: (hi + lo) * (torch.arange(hi.shape[1]) < hi.shape[1] - 32),
}
SIZES = sorted({(c[6], c[7]) for c in CASES if c[8] == 32} | {(32, 64), (1184, 736), (2048, 2048)})


@pytest.mark.parametrize("H,F", SIZES)
def test_the_bound_rejects_planted_mistakes(H, F):
    x = rows_of(40, H, 1).double()
    gu, dn = (w[0].double() for w in weights(1, F, H))
    out, b = expert(x, gu, dn, 2.0 ** -16)
    s = x @ gu.T
    h = s[:, :F] / (1.0 + torch.exp(-s[:, :F])) * s[:, F:]
    hi = h.float().bfloat16().double()
    lo = (h - hi).float().bfloat16().double()
    for name, f in MISTAKES.items():
        got = (f(hi, lo) @ dn.T).float().to(torch.bfloat16)
        assert (within(got, out, b, torch.bfloat16) <= 1.0) == (name == "none"), name


@pytest.mark.gpu
@pytest.mark.parametrize("name,counts,T,k,R,C,H,F,tile,parts", CASES, ids=IDS)
def test_expert_mlp_w4(name, counts, T, k, R, C, H, F, tile, parts):
    print(f"\n[gpu] sparse expert MLP w4 {name}", flush=True)
    assert moe.moe_expert_mlp_w4_tiling(T, k, len(counts), R, C, H, F) == (tile, parts)
    El = len(counts) // R
    L = layout_of(counts, T, k, R, C, H)
    send = rows_of(L.rows_max, H, 400 + len(name))
    gu, dn = weights(El, F, H)
    packs = [t for w in (gu, dn) for t in pack4(w.to(DEV))[0]]
    out = run(counts, T, k, R, C, H, F, L, send, packs).cpu()
    half = 2.0 ** -16 if tile == 32 else 2.0 ** -8  # of h: two bf16 parts or one
    for e, rows in some_rows(counts, 1 if sum(counts) < 300 else 7):
        want, b = expert(send[rows].double(), gu[e % El].double(), dn[e % El].double(), half)
        assert within(out[rows], want, b, torch.bfloat16) <= 1.0, e


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "w4"])
@pytest.mark.parametrize("name,T,H,E,k,F,R,C,routing", LAYER_CASES, ids=[c[0] for c in LAYER_CASES])
def test_layer(monkeypatch, name, T, H, E, k, F, R, C, routing, kind):
    print(f"\n[gpu] sparse layer {name} {kind}", flush=True)
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "w4":
        H, F = -(-H // 32) * 32, -(-F // 32) * 32
    El = E // R
    gu, dn = weights(El, F, H)
    inp = {"x": rows_of(T, H, 500 + T).to(dtype).to(DEV), "w_router": torch.zeros(E, H, device=DEV),
           "w_gate_up": gu.to(dtype).to(DEV), "w_down": dn.to(dtype).to(DEV)}
    # the logits are the biases: exact, so the routing weights' bound is a few steps of float32
    bias = torch.randn(T, E, generator=torch.Generator().manual_seed(600 + T))
    inp["bias"] = bias.to(DEV)
    packs = [t for n in ("w_gate_up", "w_down") for t in pack4(inp[n])[0]] if kind == "w4" else None
    r = Run(inp, k, R, C, packs)()
    ids = r.ids.cpu().long()
    assert torch.equal(r.logits.cpu(), bias)
    monkeypatch.setattr(ref, "expert", expert)
    want = layer(inp["x"].cpu().double(), torch.zeros(E, H, dtype=torch.float64), bias.double(), k, R, C, ids,
                 lambda l: (gu[l].double(), dn[l].double()), 0.0 if kind == "f32" else 2.0 ** -16)
    assert within(r.y.cpu(), want["y"], want["dy"], dtype) <= 1.0


@pytest.mark.gpu
def test_weights_past_4_gib():
    """The first and the last of 330 experts (4.5 GiB of gate/up codes), for the MLP and for the layer."""
    El, H, F, T = 330, 7168, 2048, 9
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    gu, dn = weights(1, F, H)
    packs = []
    for w in (gu, dn):
        (c, s), _ = pack4(w.to(DEV))
        for t in (c, s):
            full = torch.zeros((El,) + t.shape[1:], dtype=torch.uint8, device=DEV)
            full[0], full[El - 1] = t[0], t[0]
            packs.append(full)
    gu, dn = gu[0].double(), dn[0].double()
    counts = [0] * El
    counts[0], counts[El - 1] = 4, 5
    L = layout_of(counts, T, 1, 1, T, H)
    assert moe.moe_expert_mlp_w4_tiling(T, 1, El, 1, T, H, F)[0] == 32
    send = rows_of(L.rows_max, H, 21)
    out = run(counts, T, 1, 1, T, H, F, L, send, packs).cpu()
    want, b = expert(send.double(), gu, dn, 2.0 ** -16)
    assert within(out, want, b, torch.bfloat16) <= 1.0
    bias = torch.zeros(T, El)
    bias[:4, 0], bias[4:, El - 1] = 1000.0, 1000.0
    inp = {"x": send.to(DEV), "w_router": torch.zeros(El, H, device=DEV), "bias": bias.to(DEV),
           "w_down": torch.empty(0, H, F)}
    y = Run(inp, 1, 1, T, packs)().y.cpu()
    assert within(y, want, b + 8 * U * want.abs(), torch.bfloat16) <= 1.0
