"""GPU: int8 experts through the binding. Codes and scales are exact against tests/_i8_ref.py, the layout equal to
moe_dispatch's; the expert MLP is held to the float64 result of the codes it is given, within a bound counted in roundings."""
import numpy as np
import pytest
import torch

import combine_router_gemm_amd as moe
from tests._i8_ref import expert, levels
from tests._layer_ref import within
from tests.test_gpu_w4 import layout_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def scale_of(top):
    """a / 127 in float32 (numpy divides float32 correctly rounded)."""
    return torch.from_numpy(top.numpy().astype(np.float32) / np.float32(127))


def awkward(N, K, dtype, seed):
    """Rows of all sizes, with ties, zeros of both signs and far-apart values."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(N, K, generator=g) * torch.exp2(torch.randint(-130, 120, (N, 1), generator=g).float())
    w[0] = 0.0
    if N > 1:
        w[1] = torch.arange(K) % 255 - 127.0
        w[1, 0] = 254.0                      # 127 v / a is half of v: every odd value a tie
    if N > 2:
        w[2], w[2, 1] = -0.0, 1.0
    if N > 3:
        w[3] = 2.0 ** -126 * (torch.arange(K) % 3 - 1.0)
    if N > 4:
        w[4], w[4, 0], w[4, 1] = 2.0 ** -30, 3.0e38, -1.5e38
    if N > 5:
        w[5] = torch.randn(K, generator=g).round()
    return w.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 32), (33, 272), (5, 1184), (64, 2064), (9, 7168), (6, 20000), (3, 40016)])
def test_quantize_and_expand(N, K, dtype):
    print(f"\n[gpu] quantize i8 {N} {K} {dtype}", flush=True)
    w = awkward(N, K, dtype, N + K)
    q = torch.full((N, K), 99, dtype=torch.int8, device=DEV)
    s = torch.full((N,), -1.0, device=DEV)
    moe.moe_quantize_i8(w.to(DEV), q, s)
    lv, top = levels(w.double())
    assert torch.equal(q.cpu().double(), lv)
    assert torch.equal(s.cpu(), scale_of(top))
    for out_dt in (torch.float32, torch.bfloat16):
        v = torch.full((N, K), float("nan"), dtype=out_dt, device=DEV)
        moe.moe_dequantize_i8(q, s, v)
        assert torch.equal(v.cpu(), (q.cpu().float() * s.cpu().unsqueeze(1)).to(out_dt))


def test_every_bf16_ratio_rounds_to_the_nearest_level():
    """All 128 mantissas of a row's maximum against all 128 of an element at eight exponents."""
    m = 1.0 + torch.arange(128).float() / 128
    cols = torch.cat([m * 2.0 ** -e for e in range(8)])
    w = torch.cat([m.unsqueeze(1) * 2.0, cols.expand(128, -1), torch.zeros(128, 15)], 1)
    lv, top = levels(w.double())
    for dt in (torch.bfloat16, torch.float32):
        q, s = torch.empty(w.shape, dtype=torch.int8, device=DEV), torch.empty(128, device=DEV)
        moe.moe_quantize_i8(w.to(dt).to(DEV), q, s)
        assert torch.equal(q.cpu().double(), lv) and torch.equal(s.cpu(), scale_of(top))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_rows_that_are_not_finite(bad):
    w = torch.randn(40, 64, generator=torch.Generator().manual_seed(1))
    w[3, 60] = bad
    w[39] = bad
    q, s = torch.empty(40, 64, dtype=torch.int8, device=DEV), torch.empty(40, device=DEV)
    moe.moe_quantize_i8(w.to(DEV), q, s)
    assert torch.isnan(s).cpu().nonzero().reshape(-1).tolist() == [3, 39]
    assert not q[3].any() and not q[39].any()


# T, H, E, k, R, C: one launch (T <= 256) and three, capacity 0, tight and none, long rows
DISPATCH = [(1, 16, 2, 1, 1, 1), (5, 64, 8, 8, 2, 5), (256, 272, 24, 3, 3, 20), (257, 272, 24, 3, 2, 300),
            (40, 1184, 512, 8, 8, 2), (700, 7168, 16, 4, 1, 100), (30, 8208, 6, 2, 1, 30), (300, 20000, 6, 2, 1, 60),
            (33, 64, 4, 2, 1, 0), (0, 64, 4, 2, 1, 4)]


@pytest.mark.parametrize("T,H,E,k,R,C", DISPATCH)
def test_dispatch_i8(T, H, E, k, R, C):
    print(f"\n[gpu] dispatch i8 {T} {H} {E} {k} {R} {C}", flush=True)
    g = torch.Generator().manual_seed(T + H + E)
    x = (torch.randn(T, H, generator=g) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=g).float())).bfloat16()
    if T > 3:
        x[2] = 0.0
        x[3, 1] = float("nan")
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int() if T else torch.zeros(0, k).int()
    L = moe.Layout(T, k, E, R, C, H, device=DEV)
    q = torch.full((L.rows_max, H), 99, dtype=torch.int8, device=DEV)
    s = torch.full((L.rows_max,), -1.0, device=DEV)
    moe.moe_dispatch_i8(x.to(DEV), ids.to(DEV), L, q, s)
    ref = moe.Layout(T, k, E, R, C, H, device=DEV)
    send = torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_dispatch(x.to(DEV), ids.to(DEV), ref, send)
    total = int(ref.expert_offset[-1])
    for n in ("expert_count", "expert_kept", "expert_overflow", "expert_offset", "pair_row"):
        assert torch.equal(getattr(L, n), getattr(ref, n)), n
    for n in ("row_token", "row_slot"):
        assert torch.equal(getattr(L, n)[:total], getattr(ref, n)[:total]), n
    if T:
        lv, top = levels(torch.nan_to_num(x.double(), nan=0.0))
        sc = scale_of(top)
        if T > 3:
            lv[3], sc[3] = 0.0, float("nan")
        t = L.row_token[:total].cpu().long()
        assert torch.equal(q[:total].cpu().double(), lv[t])
        assert torch.equal(torch.nan_to_num(s[:total].cpu(), nan=-5.0), torch.nan_to_num(sc[t], nan=-5.0))
    assert torch.all(q[total:] == 99) and torch.all(s[total:] == -1.0)


def case(counts, T, k, R, C, H, F, seed, low=-127):
    El = len(counts) // R
    g = torch.Generator().manual_seed(seed)
    L = layout_of(counts, T, k, R, C, H)
    code = lambda *shape: torch.randint(low, 128, shape, generator=g).to(torch.int8)
    q, s = code(L.rows_max, H), torch.rand(L.rows_max, generator=g) * 0.02 + 1e-4
    weights = [code(El, 2 * F, H), torch.rand(El, 2 * F, generator=g) * 1e-3 + 1e-5, code(El, H, F),
               torch.rand(El, H, generator=g) * 1e-3 + 1e-5]
    # g of the order of one: the sums grow with the square root of H
    weights[1] /= (H / 64) ** 0.5
    return L, q, s, weights


def run(L, q, s, weights, out, **kw):
    moe.moe_expert_mlp_i8(q.to(DEV), s.to(DEV), L, *[w.to(DEV) for w in weights], out, **kw)
    return out


def check(out, q, s, weights, counts, R, every=1):
    El, at, worst = len(counts) // R, 0, 0.0
    for e, n in enumerate(counts):
        rows = list(range(at, at + n))
        rows = rows if every == 1 else sorted(set(rows[::every] + rows[-1:]))
        at += n
        if rows:
            ref, b = expert(q[rows].double(), s[rows].double(), *[w[e % El].double() for w in weights])
            worst = max(worst, within(out[rows].cpu(), ref, b, torch.bfloat16))
    return worst


CASES = [
    # name, counts, T, k, R, C, H, F, rows per tile, whether the gate/up and the down pass are split
    ("one_row", [1, 0, 0, 0], 1, 1, 1, 1, 16, 16, 32, False, False),
    ("empty", [0, 0, 0, 0], 4, 2, 1, 4, 64, 32, 32, False, False),
    ("ranks_ragged", [3, 0, 17, 1, 16, 2, 0, 15], 40, 2, 4, 17, 144, 80, 32, False, False),
    # at most eight rows: the down pass makes h's codes itself, in parts of at most 32 stages
    ("few_wide", [1, 0, 1, 0], 1, 2, 1, 1, 272, 8208, 32, False, True),
    ("few_ranks", [1, 0, 2, 0, 0, 1, 1, 0, 1, 0, 0, 2], 4, 2, 3, 4, 1040, 1424, 32, False, False),
    ("few_tall", [8, 0], 8, 1, 1, 8, 2064, 4112, 32, True, True),
    ("nine", [9, 0], 9, 1, 1, 9, 2064, 4112, 32, True, True),
    ("rows_16_32", [16, 33, 32, 31], 64, 2, 1, 33, 544, 288, 32, False, False),
    ("wide", [9, 23], 32, 1, 1, 32, 1184, 736, 32, False, False),
    # few tiles and a wide K: a pass is split, its last part shorter; with two ranks
    ("split_down", [9, 0, 32, 1], 42, 1, 1, 42, 160, 4304, 32, False, True),
    ("split_down_ranks", [3, 16, 0, 1, 7, 20], 47, 1, 2, 20, 64, 4160, 32, False, True),
    ("split_gate_up", [9, 0, 32, 1], 42, 1, 1, 42, 4304, 160, 32, True, False),
    ("split_gate_up_ranks", [3, 16, 0, 1, 7, 20], 47, 1, 2, 20, 4160, 48, 32, True, False),
    ("split_both", [1, 1], 2, 1, 1, 1, 2064, 2320, 32, True, True),
    ("tile_64", [64, 130, 1, 61], 256, 1, 1, 256, 4112, 4112, 64, False, False),
    ("tile_64_ranks", [40, 24, 1, 33, 0, 34, 50, 66], 256, 1, 2, 70, 4112, 2064, 64, False, False),
    ("tile_128", [300, 129, 1, 513] * 3, 2829, 1, 1, 700, 1184, 736, 128, False, False),
    ("tile_128_ranks", [128, 1, 0, 127, 33, 200, 256, 255] * 3, 3000, 1, 2, 300, 1184, 736, 128, False, False),
    ("tile_256", [1025, 700, 256, 255] * 3, 6708, 1, 1, 6708, 1184, 736, 256, False, False),
    ("tile_256_ranks", [257, 255, 256, 1, 1400, 0, 700, 33] * 2, 6000, 1, 2, 6000, 1040, 720, 256, False, False),
]


@pytest.mark.parametrize("name,counts,T,k,R,C,H,F,rows,gu,dn", CASES, ids=[c[0] for c in CASES])
def test_expert_mlp_i8(name, counts, T, k, R, C, H, F, rows, gu, dn):
    print(f"\n[gpu] expert MLP i8 {name}", flush=True)
    tiling = moe.moe_expert_mlp_i8_tiling(T, k, len(counts), R, C, H, F)
    assert (tiling[0], tiling[1] > 1, tiling[2] > 1) == (rows, gu, dn)
    L, q, s, weights = case(counts, T, k, R, C, H, F, 100 + len(name))
    n = moe.moe_expert_mlp_i8_workspace_bytes(T, k, len(counts), R, C, H, F)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    out = run(L, q, s, weights, torch.full((L.rows_max, H), -7.0, dtype=torch.bfloat16, device=DEV), workspace=ws)
    total = sum(counts)
    assert torch.all(out[total:] == -7.0)  # rows past the kept ones are left alone
    assert check(out, q, s, weights, counts, R, 1 if total < 300 else 23) <= 1.0
    ws.fill_(0x11)
    again = run(L, q, s, weights, torch.full_like(out, -7.0), workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_largest_sums_do_not_overflow():
    """Every code -128 or 127 at the longest K: the sum is within 2^18 of 2^31."""
    H, F = 131056, 16
    L, q, s, weights = case([2], 2, 1, 1, 2, H, F, 3)
    q.fill_(-128)
    weights[0].fill_(-128)
    weights[0][0, 1::2] = 127
    weights[1].fill_(1e-6)
    s.fill_(1e-4)
    out = run(L, q, s, weights, torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV))
    assert check(out, q, s, weights, [2], 1) <= 1.0
    L, q, s, weights = case([2], 2, 1, 1, 2, 16, 131056, 4)
    weights[2].fill_(-128)
    out = run(L, q, s, weights, torch.zeros(L.rows_max, 16, dtype=torch.bfloat16, device=DEV))
    assert check(out, q, s, weights, [2], 1) <= 1.0


@pytest.mark.parametrize("counts,T", [([5, 20, 3, 0], 28), ([200, 150, 3, 0], 600), ([700, 600], 1300)])
def test_rows_that_are_not_finite_stay_apart(counts, T):
    H, F, R = 96, 64, 1
    L, q, s, weights = case(counts, T, 1, R, T, H, F, 9)
    good = run(L, q, s, weights, torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV))
    s[6] = float("nan")
    s[2] = float("inf")
    weights[1][1, 3] = float("inf")  # an expert's gate channel: all of its rows
    out = run(L, q, s, weights, torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV))
    nan = torch.isnan(out.float()).all(dim=1).cpu()
    bad = set(range(counts[0], counts[0] + counts[1])) | {2, 6}
    assert nan.nonzero().reshape(-1).tolist() == sorted(bad)
    keep = [r for r in range(sum(counts)) if r not in bad]
    assert torch.equal(out[keep], good[keep])


def test_zero_rows_and_zero_channels():
    L, q, s, weights = case([6, 3], 9, 1, 1, 9, 64, 48, 11)
    q[2] = 0
    s[4] = 0.0
    weights[0][1] = 0
    weights[3][0, 5] = 0.0
    out = run(L, q, s, weights, torch.full((L.rows_max, 64), -7.0, dtype=torch.bfloat16, device=DEV))
    assert not out[2].any() and not out[4].any() and not out[6:9].any() and not out[:6, 5].any()
    assert check(out, q, s, weights, [6, 3], 1) <= 1.0


def test_graph_side_stream_and_shared_workspace():
    counts = [20, 7, 0, 33]
    L, q, s, weights = case(counts, 60, 1, 1, 40, 160, 4304, 10)
    args = [q.to(DEV), s.to(DEV), L] + [w.to(DEV) for w in weights]
    out = torch.zeros(L.rows_max, 160, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(moe.moe_expert_mlp_i8_workspace_bytes(60, 1, 4, 1, 40, 160, 4304), dtype=torch.uint8, device=DEV)
    moe.moe_expert_mlp_i8(*args, out, workspace=ws)
    ref = out.clone()
    other = [(q.to(DEV) // 2), *args[1:]]
    out2 = torch.zeros_like(out)
    moe.moe_expert_mlp_i8(*other, out2, workspace=ws)
    ref2 = out2.clone()
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    moe.moe_expert_mlp_i8(*args, out, stream=side)  # its own workspace, on another stream
    junk = torch.full((ws.numel(),), 0xA5, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and junk[0] == 0xA5
    graphs = []
    for a, o in ((args, out), (other, out2)):  # two graphs that share the workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_expert_mlp_i8(*a, o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        out.zero_()
        out2.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(out2, ref2)
        ws.fill_(0x3C)
        torch.cuda.synchronize()


def test_weights_past_4_gib():
    El, H, F, T = 330, 7168, 1024, 9  # 4.5 GiB of gate/up codes
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    counts = [0] * El
    counts[0], counts[El - 1] = 4, 5
    L = layout_of(counts, T, 1, 1, T, H)
    g = torch.Generator(device=DEV).manual_seed(5)
    code = lambda *shape: torch.randint(-127, 128, shape, dtype=torch.int8, device=DEV, generator=g)
    weights = [code(El, 2 * F, H), torch.full((El, 2 * F), 1e-4, device=DEV), code(El, H, F),
               torch.full((El, H), 1e-4, device=DEV)]
    q, s = code(T, H), torch.full((T,), 1e-3, device=DEV)
    out = torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_mlp_i8(q, s, L, *weights, out)
    for l, rows in ((0, slice(0, 4)), (El - 1, slice(4, 9))):
        ref, b = expert(q[rows].cpu().double(), s[rows].cpu().double(), *[w[l].cpu().double() for w in weights])
        assert within(out[rows].cpu(), ref, b, torch.bfloat16) <= 1.0


def test_rows_past_4_gib_of_h():
    """h of 66000 rows x 17008 columns is past 4 GiB in float32, its codes past 1 GiB."""
    rows, H, F = 66000, 32, 17008
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB")
    L, q, s, weights = case([rows - 300, 300], rows, 1, 1, rows, H, F, 21)
    out = run(L, q, s, weights, torch.zeros(L.rows_max, H, dtype=torch.bfloat16, device=DEV))
    pick = list(range(0, 40)) + list(range(rows - 330, rows))
    for e, sel in ((0, [r for r in pick if r < rows - 300]), (1, [r for r in pick if r >= rows - 300])):
        ref, b = expert(q[sel].double(), s[sel].double(), *[w[e].double() for w in weights])
        assert within(out[sel].cpu(), ref, b, torch.bfloat16) <= 1.0


def test_more_tokens_than_a_launch_holds_in_one_direction():
    """2^24 workgroups of 256 threads are 2^32 threads. Rows and layout against the row kernel and moe_dispatch."""
    T, H, E, k, C = (1 << 24) + 5, 16, 3, 1, 1 << 24
    print(f"\n[gpu] dispatch i8 and combine backward {T} {H}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    ids = torch.randint(0, E, (T, k), device=DEV, generator=g, dtype=torch.int32)
    L, ref = moe.Layout(T, k, E, 1, C, H, device=DEV), moe.Layout(T, k, E, 1, C, H, device=DEV)
    q, s = torch.empty(L.rows_max, H, dtype=torch.int8, device=DEV), torch.empty(L.rows_max, device=DEV)
    moe.moe_dispatch_i8(x, ids, L, q, s)
    send = torch.empty(L.rows_max, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_dispatch(x, ids, ref, send)
    assert torch.equal(L.pair_row, ref.pair_row) and torch.equal(L.row_token, ref.row_token)
    want_q, want_s = torch.empty_like(q), torch.empty_like(s)
    moe.moe_quantize_i8(send, want_q, want_s)
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    w, d_w = torch.rand(T, k, device=DEV, generator=g), torch.full((T, k), -9.0, device=DEV)
    d_out = torch.empty_like(send)
    moe.moe_combine_backward(x, send, L, w, d_w, d_out_buf=d_out)
    # every product is of equal values: sums of H squares, each addition off by half a step of the sum at most
    exact = (x.double() ** 2).sum(1)
    assert bool(((d_w[:, 0].double() - exact).abs() <= H * 2.0 ** -24 * exact).all())
    assert torch.equal(d_out[L.pair_row[:, 0].long()], (w * x.float()).bfloat16())


def test_binding_refusals():
    L, q, s, weights = case([3, 2], 5, 1, 1, 5, 64, 32, 2)
    args = [q.to(DEV), s.to(DEV)] + [w.to(DEV) for w in weights]
    out = torch.zeros(L.rows_max, 64, dtype=torch.bfloat16, device=DEV)
    call = lambda a, o=out, lay=L, **kw: moe.moe_expert_mlp_i8(a[0], a[1], lay, *a[2:], o, **kw)
    swap = lambda i, t: args[:i] + [t] + args[i + 1:]
    for bad in (swap(0, args[0].float()), swap(0, args[0][:, :32].contiguous()), swap(1, args[1].double()),
                swap(2, args[2].transpose(0, 1)), swap(3, args[3][:1]), swap(4, args[4].cpu()), swap(5, args[5][:, :3])):
        with pytest.raises(moe.MoeError):
            call(bad)
    with pytest.raises(moe.MoeError):
        call(args, out.float())
    with pytest.raises(moe.MoeError):
        call(args, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    host = layout_of([3, 2], 5, 1, 1, 5, 64)
    host.expert_kept = host.expert_kept.cpu()
    with pytest.raises(moe.MoeError):
        call(args, lay=host)
