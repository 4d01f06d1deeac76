"""GPU: 4-bit expert weights through the C ABI. Quantisation and expansion are bit-exact against oracle/w4.py; the
expert MLP is held to the float64 result of the values its codes stand for (bounds: tests/_layer_ref.py)."""
import numpy as np
import pytest
import torch

import combine_router_gemm_amd as moe
import oracle
from tests._layer_ref import expert, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def packed(N, K, lead=(), device=DEV):
    cs, ss = moe.moe_w4_shapes(*lead, N, K)
    return torch.full(cs, 0xEE, dtype=torch.uint8, device=device), torch.full(ss, 0xEE, dtype=torch.uint8, device=device)


def weights(N, K, dtype, seed, spread=3):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(N, K, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (N, K // 32), generator=g)
                                                   .float()).repeat_interleave(32, 1)
    return w.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(16, 32), (16, 96), (48, 512), (32, 544), (112, 1184)])
def test_quantize_and_expand_match_the_oracle(N, K, dtype):
    w = weights(N, K, dtype, N * 7 + K)
    # ties, zeros of both signs, a group of zeros, the clamps of the scale, borders of the group maximum
    w[0, :8] = torch.tensor([6.0, 0.25, -0.75, 1.25, -1.75, 2.5, 3.5, -5.0])
    w[1, :32] = 0.0
    w[2, :32], w[2, 3] = 0.0, -0.0
    w[3, :32] = 2.0 ** -126
    w[4, 0] = 3.0e38
    w[5, :32] = 0.0
    w[5, 0] = 1.5
    w[6, :32] = 0.0
    w[6, 0] = 1.5 + 2.0 ** -7
    codes, scales = packed(N, K)
    moe.moe_quantize_w4(w.to(DEV), codes, scales)
    c_ref, s_ref = oracle.w4.quantize(w.double().numpy())
    tc, ts = oracle.w4.pack(c_ref, s_ref)
    assert np.array_equal(codes.cpu().numpy(), tc)
    assert np.array_equal(scales.cpu().numpy(), ts)
    for out_dt in (torch.float32, torch.bfloat16):
        v = torch.full((N, K), float("nan"), dtype=out_dt, device=DEV)
        moe.moe_dequantize_w4(codes, scales, v)
        assert np.array_equal(v.double().cpu().numpy(), oracle.w4.values(c_ref, s_ref))


def test_every_code_at_every_scale_expands_exactly():
    # 16 codes x scales 7 .. 252, one scale per group
    N, K = 16, 512
    codes = np.tile(np.arange(16, dtype=np.uint8), (N, K // 16))
    scales = (7 + np.arange(N * K // 32) % 246).astype(np.uint8).reshape(N, K // 32)
    tc, ts = oracle.w4.pack(codes, scales)
    for dt in (torch.float32, torch.bfloat16):
        v = torch.empty(N, K, dtype=dt, device=DEV)
        moe.moe_dequantize_w4(torch.from_numpy(tc).to(DEV), torch.from_numpy(ts).to(DEV), v)
        assert np.array_equal(v.double().cpu().numpy(), oracle.w4.values(codes, scales))


def test_batched_matrices_follow_one_another():
    w = torch.stack([weights(32, 160, torch.bfloat16, 50 + i) for i in range(3)]).to(DEV)
    codes, scales = packed(32, 160, (3,))
    moe.moe_quantize_w4(w, codes, scales)
    for i in range(3):
        c1, s1 = packed(32, 160)
        moe.moe_quantize_w4(w[i], c1, s1)
        assert torch.equal(codes[i], c1) and torch.equal(scales[i], s1)


def layout_of(counts, T, k, R, C, H):
    """A layout whose experts hold counts[e] rows (row_token and pair_row are not read by the expert MLP)."""
    E = len(counts)
    L = moe.Layout(T, k, E, R, C, H, device=DEV)
    kept = torch.tensor(counts, dtype=torch.int32)
    assert int(kept.max()) <= C and int(kept.sum()) <= L.rows_max
    L.expert_kept.copy_(kept)
    L.expert_offset.copy_(torch.cat([torch.zeros(1, dtype=torch.int64), kept.cumsum(0)]).int())
    for n in ("expert_count", "expert_overflow", "row_token", "row_slot", "pair_row"):
        getattr(L, n).zero_()
    return L


def case(counts, T, k, R, C, H, F, seed):
    E, El = len(counts), len(counts) // R
    g = torch.Generator().manual_seed(seed)
    L = layout_of(counts, T, k, R, C, H)
    send = torch.randn(L.rows_max, H, generator=g).to(torch.bfloat16)
    gu = torch.randn(El, 2 * F, H, generator=g).mul_(0.05).to(torch.bfloat16)
    dn = torch.randn(El, H, F, generator=g).mul_(0.05).to(torch.bfloat16)
    packs, vals = [], []
    for w in (gu, dn):
        c, s = packed(w.shape[1], w.shape[2], (El,))
        moe.moe_quantize_w4(w.to(DEV), c, s)
        v = torch.empty_like(w, device=DEV)
        moe.moe_dequantize_w4(c, s, v)
        packs += [c, s]
        vals.append(v.cpu().double())
    return L, send, packs, vals


def check_rows(out, L, send, vals, counts, R, every=1):
    E, El = len(counts), len(counts) // R
    at, worst = 0, 0.0
    for e in range(E):
        n = counts[e]
        rows = list(range(at, at + n))
        rows = rows if every == 1 else sorted(set(rows[::every] + rows[-1:]))
        if rows:
            ref, b = expert(send[rows].double(), vals[0][e % El], vals[1][e % El], 2.0 ** -8)
            worst = max(worst, within(out[rows].cpu(), ref, b, torch.bfloat16))
        at += n
    return worst


CASES = [
    # name, counts, T, k, R, C, H, F
    ("one_row", [1, 0, 0, 0], 1, 1, 1, 1, 32, 32),
    ("empty", [0, 0, 0, 0], 4, 2, 1, 4, 64, 32),
    ("ranks_ragged", [3, 0, 17, 1, 16, 2, 0, 15], 40, 2, 4, 17, 160, 96),
    ("rows_16_32", [16, 33, 32, 31], 64, 2, 1, 33, 544, 288),
    ("tiles_64", [64, 65, 1, 130, 0, 63], 190, 2, 2, 190, 256, 160),
    ("wide", [9, 23], 32, 1, 1, 32, 1184, 736),
    ("many_rows", [300, 129, 1, 513], 513, 2, 1, 513, 288, 352),
    ("many_rows_ranks", [257, 255, 256, 1, 400, 0], 700, 2, 3, 500, 640, 256),
    ("tall", [1500, 1025], 1500, 2, 1, 1500, 96, 160),
    # F much wider than H and few tiles: the down pass splits its K, unevenly; with two ranks
    ("split", [9, 0, 32, 1], 42, 1, 1, 42, 160, 2304),
    ("split_ranks", [3, 16, 0, 1, 7, 20], 47, 1, 2, 20, 64, 4160),
    ("split_many_rows", [150, 70], 220, 1, 1, 220, 96, 4160),
    # many tiles (tests/test_w4_tiles.py has the cases of the 128- and 256-row tiles)
    ("tile_128", [640, 129, 0, 1, 257, 500, 64, 33], 2560, 2, 1, 2560, 288, 2016),
    ("tile_256_ranks", [512, 1, 0, 300, 255, 17, 128, 33, 256, 0, 31, 90, 1, 700, 64, 129], 2048, 2, 2, 2048, 160, 2016),
]


@pytest.mark.parametrize("name,counts,T,k,R,C,H,F", CASES, ids=[c[0] for c in CASES])
def test_expert_mlp_w4(name, counts, T, k, R, C, H, F):
    print(f"\n[gpu] expert MLP w4 {name}", flush=True)
    L, send, packs, vals = case(counts, T, k, R, C, H, F, 100 + len(name))
    out = torch.full((L.rows_max, H), -7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((moe.moe_expert_mlp_w4_workspace_bytes(T, k, len(counts), R, C, F),), 0xFF, dtype=torch.uint8,
                    device=DEV)
    moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out, workspace=ws)
    total = sum(counts)
    assert torch.all(out[total:] == -7.0)  # rows past the kept ones are left alone
    assert check_rows(out, L, send, vals, counts, R, 1 if total < 300 else 7) <= 1.0
    again = torch.full_like(out, -7.0)
    ws.fill_(0x11)
    moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, again, workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_expert_mlp_w4_keeps_non_finite_rows_apart():
    counts = [5, 20, 3, 0]
    L, send, packs, vals = case(counts, 28, 1, 1, 28, 96, 64, 9)
    send[6, 3] = float("inf")
    send[27, 0] = float("nan")
    out = torch.zeros(L.rows_max, 96, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out)
    bad = ~torch.isfinite(out.float()).all(dim=1).cpu()
    assert bad[6] and bad[27] and int(bad.sum()) == 2


def test_expert_mlp_w4_infinite_h_stays_infinite():
    counts, H, F = [2, 20], 32, 32
    L, send, _, _ = case(counts, 22, 1, 1, 22, H, F, 12)
    send.fill_(1.0)
    gu = torch.zeros(2, 2 * F, H, dtype=torch.bfloat16, device=DEV)
    gu[:, 3, 0] = gu[:, F + 3, 0] = 2.0 ** 100
    packs = []
    for w in (gu, torch.ones(2, H, F, dtype=torch.bfloat16, device=DEV)):
        c, s = packed(w.shape[1], w.shape[2], (2,))
        moe.moe_quantize_w4(w, c, s)
        packs += [c, s]
    out = torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out)
    assert torch.all(out[:22] == float("inf"))


def test_expert_mlp_w4_graph_and_side_stream():
    counts = [20, 7, 0, 33]
    L, send, packs, _ = case(counts, 40, 2, 1, 40, 160, 96, 10)
    send = send.to(DEV)
    out = torch.zeros(L.rows_max, 160, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(moe.moe_expert_mlp_w4_workspace_bytes(40, 2, 4, 1, 40, 96), dtype=torch.uint8, device=DEV)
    moe.moe_expert_mlp_w4(send, L, *packs, out, workspace=ws)
    ref = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    moe.moe_expert_mlp_w4(send, L, *packs, out, stream=side)  # its own workspace, on another stream
    junk = torch.full((ws.numel(),), 0xA5, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and junk[0] == 0xA5
    with torch.cuda.stream(side):
        moe.moe_expert_mlp_w4(send, L, *packs, out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_expert_mlp_w4(send, L, *packs, out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        ws.fill_(0x3C)


def test_expert_mlp_w4_weights_past_4_gib():
    El, H, F, T = 330, 7168, 2048, 9  # 4.5 GiB of gate/up codes
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    counts = [0] * El
    counts[0], counts[El - 1] = 4, 5
    L = layout_of(counts, T, 1, 1, T, H)
    g = torch.Generator(device=DEV).manual_seed(5)
    packs = []
    for N, K in ((2 * F, H), (H, F)):
        cs, ss = moe.moe_w4_shapes(El, N, K)
        packs += [torch.randint(0, 256, cs, dtype=torch.uint8, device=DEV, generator=g),
                  torch.randint(118, 122, ss, dtype=torch.uint8, device=DEV, generator=g)]
    send = torch.randn(L.rows_max, H, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    out = torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_mlp_w4(send.to(DEV), L, *packs, out)
    for l, rows in ((0, slice(0, 4)), (El - 1, slice(4, 9))):
        v = []
        for (N, K), c, s in (((2 * F, H), *packs[:2]), ((H, F), *packs[2:])):
            w = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
            moe.moe_dequantize_w4(c[l], s[l], w)
            v.append(w.double().cpu())
        ref, b = expert(send[rows].double(), v[0], v[1], 2.0 ** -8)
        assert within(out[rows].cpu(), ref, b, torch.bfloat16) <= 1.0
