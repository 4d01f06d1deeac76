"""GPU: balance loss, combine backward and router backward through the binding against tests/_router_ref.py (float64, bounds
counted in roundings), and a run of them together with the int8 experts."""
import pytest
import torch

import combine_router_gemm_amd as moe
from tests._layer_ref import U, within
from tests._router_ref import balance, combine_backward, route_backward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def top_ids(logits, k):
    return torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k].int().contiguous()


def run_balance(logits, ids, weight, offset=None, mask=None, grad=True, **kw):
    T, E = logits.shape
    S = 1 if offset is None else len(offset) - 1
    loss = torch.full((1,), -9.0, device=DEV)
    count = torch.full((S, E), -9, dtype=torch.int32, device=DEV)
    d = torch.full((T, E), -9.0, device=DEV) if grad else None
    off = None if offset is None else torch.tensor(offset, dtype=torch.int32, device=DEV)
    moe.moe_balance_loss(logits.to(DEV), ids.to(DEV), weight, loss, count, d_logits=d, seq_offset=off,
                         token_mask=None if mask is None else mask.to(DEV), **kw)
    return loss, count, d


def check_balance(logits, ids, weight, offset=None, mask=None):
    loss, count, d = run_balance(logits, ids, weight, offset, mask)
    r = balance(logits.double(), ids, weight, offset, mask)
    assert torch.equal(count.cpu().long(), r["count"])
    # weight is a float32
    assert abs(float(loss) - r["loss"]) <= r["dloss"] + 4 * U * abs(r["loss"]) + 1e-44
    assert within(d.cpu(), r["d"], r["db"] + 2 * U * r["d"].abs(), F32) <= 1.0
    return loss, count, d


# T, E, k: groups of 4, 16 and 64 lanes, vectors and single logits, many workgroups
@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (1, 1, 1), (7, 8, 8), (33, 15, 3), (64, 24, 3), (100, 61, 4), (65, 65, 2),
                                   (50, 128, 1), (40, 129, 8), (301, 256, 8), (19, 260, 5), (23, 384, 8), (9, 509, 8),
                                   (17, 512, 8), (5000, 12, 2)])
def test_balance_one_sequence(T, E, k):
    print(f"\n[gpu] balance {T} {E} {k}", flush=True)
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=g) * 3 - 0.5 * torch.arange(E).float() / E
    check_balance(logits, top_ids(logits, k), 0.01)


@pytest.mark.parametrize("offset", [[0, 50, 50, 51, 200], [3, 40, 40, 180], [0, 0, 0], [200, 200], [0, 200], [7, 8],
                                    list(range(0, 201, 5)), [0, 100, 190] + [190] * 20])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_sequences(offset, masked):
    print(f"\n[gpu] balance {offset[:6]} {masked}", flush=True)
    g = torch.Generator().manual_seed(len(offset))
    logits = torch.randn(200, 24, generator=g) * 2
    mask = (torch.rand(200, generator=g) < 0.7).to(torch.uint8) if masked else None
    if masked:
        mask[40:60] = 0
    _, _, d = check_balance(logits, top_ids(logits, 3), 1.0, offset, mask)
    idle = [t for t in range(200) if not (offset[0] <= t < offset[-1]) or (masked and not mask[t])]
    assert not d[idle].any()


def test_balance_many_sequences_of_a_large_batch():
    g = torch.Generator().manual_seed(3)
    T = 3000
    logits = torch.randn(T, 16, generator=g)
    cuts = sorted(torch.randint(0, T, (70,), generator=g).tolist())
    check_balance(logits, top_ids(logits, 2), 0.5, [0] + cuts + [T - 11], torch.rand(T, generator=g) < 0.9)


def test_balance_of_an_even_router_is_its_weight():
    loss, count, d = run_balance(torch.zeros(64, 8), torch.arange(128).view(64, 2).int() % 8, 0.25)
    assert float(loss) == 0.25 and torch.all(count == 16) and not d.any()


@pytest.mark.parametrize("T,E,offset", [(100, 6, None), (70, 8, None), (33, 1, None), (90, 8, [0, 11, 40, 40, 85]),
                                        (60, 5, list(range(0, 61, 5)))])
def test_balance_gradient_of_even_choices_is_zero(T, E, offset):
    """Every expert chosen by every token (k = E): the gradient is 0, not what is left of a difference of roundings."""
    print(f"\n[gpu] balance even {T} {E} {offset}", flush=True)
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=g) * 3
    ids = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).int()
    S = 1 if offset is None else len(offset) - 1
    loss, count = torch.empty(1, device=DEV), torch.empty(S, E, dtype=torch.int32, device=DEV)
    d = torch.full((T, E), -9.0, device=DEV)
    off = None if offset is None else torch.tensor(offset, dtype=torch.int32, device=DEV)
    moe.moe_balance_loss(logits.to(DEV), ids.to(DEV), 0.25, loss, count, d_logits=d, seq_offset=off)
    assert not d.any()
    # f = 1 / E and the sum of p is 1, both rounded a few times: the factors and the softmax take some ten roundings
    assert abs(float(loss) - 0.25) < 0.25 * 16 * 2.0 ** -24


def test_balance_padding_and_masked_experts():
    """What a masked token holds does not matter; -inf logits have p = 0; a row of them adds nothing; ids out of range are not
    counted; a NaN of a counted token shows."""
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(40, 12, generator=g)
    ids = top_ids(logits, 2)
    mask = torch.ones(40, dtype=torch.uint8)
    mask[[3, 39]] = 0
    logits[3], logits[39] = float("nan"), float("inf")
    logits[5, 4:], logits[6] = -float("inf"), -float("inf")
    logits[7, :11] = torch.finfo(F32).min
    logits[8] = torch.finfo(F32).max
    ids[10, 0], ids[11, 1] = -1, 12
    check_balance(logits, ids, 0.1, None, mask)
    logits[20, 1] = float("nan")
    loss, _, d = run_balance(logits, ids, 0.1, None, mask)
    assert torch.isnan(loss) and torch.isnan(d[20]).all() and not torch.isnan(d[:20]).any()


def test_balance_without_tokens_or_gradient():
    loss, count, _ = run_balance(torch.zeros(0, 8), torch.zeros(0, 2, dtype=torch.int32), 1.0, [0, 0, 0])
    assert float(loss) == 0 and not count.any()
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(300, 20, generator=g)
    a = run_balance(logits, top_ids(logits, 3), 0.1)
    b = run_balance(logits, top_ids(logits, 3), 0.1, grad=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_balance_offsets_out_of_range_stay_in_bounds():
    """Offsets beyond the batch, negative or decreasing: what is counted is unspecified, nothing else is touched."""
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(50, 8, generator=g)
    for off in ([-5, 20, 1000], [40, 10, 30], [1 << 30, -(1 << 30), 7]):
        loss, count, d = run_balance(logits, top_ids(logits, 2), 1.0, off)
        assert int(count.min()) >= 0 and torch.isfinite(d).all() and torch.isfinite(loss).all()


def layout(ids, E, C, H):
    T, k = ids.shape
    L = moe.Layout(T, k, E, 1, C, H, device=DEV)
    moe.moe_dispatch(torch.zeros(T, H, dtype=BF16, device=DEV), ids.to(DEV), L,
                     torch.zeros(L.rows_max, H, dtype=BF16, device=DEV))
    return L


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H,E,k,C", [(1, 8, 1, 1, 1), (5, 16, 4, 4, 5), (40, 72, 8, 2, 7), (33, 1184, 24, 8, 6),
                                       (20, 2056, 6, 3, 20), (9, 7168, 16, 8, 9), (7, 9000, 5, 2, 3), (30, 64, 4, 2, 0)])
def test_combine_backward(T, H, E, k, C, dtype):
    print(f"\n[gpu] combine backward {T} {H} {E} {k} {C} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T + H)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    L = layout(ids, E, C, H)
    dy = torch.randn(T, H, generator=g).to(dtype)
    out = torch.randn(L.rows_max, H, generator=g).to(dtype)
    total = int(L.expert_offset[-1])
    out[total:] = float("nan")
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    d_w = torch.full((T, k), -9.0, device=DEV)
    d_out = torch.full((L.rows_max, H), -9.0, dtype=dtype, device=DEV)
    moe.moe_combine_backward(dy.to(DEV), out.to(DEV), L, w.to(DEV), d_w, d_out_buf=d_out)
    r = combine_backward(dy.double(), out.double(), L.pair_row.cpu(), w.double())
    assert within(d_w.cpu(), r[0], r[1], F32) <= 1.0
    assert within(d_out[:total].cpu(), r[2][:total], r[3][:total], dtype) <= 1.0
    assert torch.all(d_out[total:] == -9.0)
    alone = torch.full((T, k), -9.0, device=DEV)
    moe.moe_combine_backward(dy.to(DEV), out.to(DEV), L, w.to(DEV), alone)
    assert torch.equal(alone, d_w)


def test_dispatch_gradient_is_the_combine_with_weights_of_one():
    g = torch.Generator().manual_seed(5)
    T, H, E, k, C = 30, 64, 6, 3, 9
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    L = layout(ids, E, C, H)
    d_send = torch.randn(L.rows_max, H, generator=g)
    d_x = torch.empty(T, H, device=DEV)
    moe.moe_combine(d_send.to(DEV), L, torch.ones(T, k, device=DEV), d_x)
    row = L.pair_row.cpu()
    ref = torch.stack([sum((d_send[r].double() for r in row[t].tolist() if r >= 0), torch.zeros(H).double())
                       for t in range(T)])
    assert torch.allclose(d_x.cpu().double(), ref, rtol=0, atol=3 * U * 3 * 8)


ROUTE = [(1, 8, 1, 1), (3, 64, 8, 2), (64, 128, 24, 3), (65, 264, 61, 4), (129, 1184, 130, 8), (300, 72, 512, 8),
         (1000, 512, 16, 2), (257, 2048, 256, 8), (2100, 136, 40, 5)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H,E,k", ROUTE)
def test_route_backward(T, H, E, k, dtype):
    print(f"\n[gpu] route backward {T} {H} {E} {k} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T + H + E)
    x = torch.randn(T, H, generator=g).to(dtype)
    wr = torch.randn(E, H, generator=g) * 0.05
    lg = torch.randn(T, E, generator=g)
    ids = top_ids(lg, k)
    w = torch.softmax(torch.gather(lg, 1, ids.long()), 1)
    d_w, d_in = torch.randn(T, k, generator=g), torch.randn(T, E, generator=g) * 0.1
    new = lambda *s, dt=F32: torch.full(s, -9.0, dtype=dt, device=DEV)
    code = moe.MOE_BF16 if dtype is BF16 else moe.MOE_F32
    n = moe.moe_route_backward_workspace_bytes(T, H, E, code)
    for use_w, use_in in ((True, True), (True, False), (False, True)):
        got = dict(d_logits=new(T, E), d_x=new(T, H, dt=dtype), d_w_router=new(E, H), d_bias=new(E))
        dev = [t.to(DEV) for t in (x, wr, ids, w)]
        a, b = d_w.to(DEV) if use_w else None, d_in.to(DEV) if use_in else None
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
        moe.moe_route_backward(*dev, a, b, got["d_logits"], d_x=got["d_x"], d_w_router=got["d_w_router"],
                               d_bias=got["d_bias"], workspace=ws)
        r = route_backward(x.double(), wr.double(), ids.long(), w.double(), d_w.double() if use_w else None,
                           d_in.double() if use_in else None, dtype is BF16)
        for name, (ref, bound) in r.items():
            assert within(got[name].cpu(), ref, bound, got[name].dtype) <= 1.0, name
    # each output alone equals all of them together; d_logits in place; bits do not depend on the workspace's contents
    for name in ("d_x", "d_w_router", "d_bias"):
        one, dl = torch.full_like(got[name], -9.0), d_in.to(DEV)
        moe.moe_route_backward(*dev, None, dl, dl, **{name: one},
                               workspace=torch.full((n,), 0x11, dtype=torch.uint8, device=DEV))
        assert torch.equal(one, got[name]) and torch.equal(dl, got["d_logits"])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_backward_wide_ranges(dtype):
    """Gradients and weights over many powers of two: each sum is held to the sum of its terms' sizes."""
    g = torch.Generator().manual_seed(77)
    T, H, E, k = 150, 264, 24, 3
    spread = lambda *s: torch.randn(*s, generator=g) * torch.exp2(torch.randint(-30, 20, s, generator=g).float())
    x, wr, d_in = spread(T, H).to(dtype), spread(E, H), spread(T, E)
    lg = torch.randn(T, E, generator=g)
    ids = top_ids(lg, k)
    w = torch.softmax(torch.gather(lg, 1, ids.long()), 1)
    got = dict(d_logits=torch.empty(T, E, device=DEV), d_x=torch.empty(T, H, dtype=dtype, device=DEV),
               d_w_router=torch.empty(E, H, device=DEV), d_bias=torch.empty(E, device=DEV))
    moe.moe_route_backward(x.to(DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), None, d_in.to(DEV), got["d_logits"],
                           d_x=got["d_x"], d_w_router=got["d_w_router"], d_bias=got["d_bias"])
    r = route_backward(x.double(), wr.double(), ids.long(), w.double(), None, d_in.double(), dtype is BF16)
    for name, (ref, bound) in r.items():
        assert within(got[name].cpu(), ref, bound, got[name].dtype) <= 1.0, name


def test_route_backward_of_tiny_and_huge_tokens():
    """Tokens and columns whose size is far from one (subnormal gradients among them): fp16's powers of two are each's own."""
    g = torch.Generator().manual_seed(31)
    T, H, E = 70, 264, 24
    rows = torch.tensor([-140.0, -126.0, -100.0, -60.0, 0.0, 60.0, 90.0])[torch.arange(T) % 7].unsqueeze(1)
    cols = torch.tensor([-30.0, -20.0, 0.0, 20.0, 30.0, -126.0])[torch.arange(H) % 6]
    d_in = (torch.randn(T, E, generator=g).double() * torch.exp2(rows.double())).float()
    d_in[5] = 0.0
    wr = (torch.randn(E, H, generator=g).double() * torch.exp2(cols.double())).float()
    wr[:, 7] = 0.0
    x = torch.randn(T, H, generator=g).to(BF16)
    d_x = torch.empty(T, H, dtype=BF16, device=DEV)
    ids, w = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
    moe.moe_route_backward(x.to(DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), None, d_in.to(DEV), torch.empty(T, E, device=DEV),
                           d_x=d_x)
    ref, bound = route_backward(x.double(), wr.double(), ids.long(), w.double(), None, d_in.double(), True)["d_x"]
    # float32 sums of the scaled products are exact to U; a result that is subnormal in bf16 is off by half its step there
    assert within(d_x.cpu(), ref, bound + 2.0 ** -134, BF16) <= 1.0


def test_route_backward_non_finite_stays_apart():
    g = torch.Generator().manual_seed(32)
    T, H, E = 40, 136, 12
    for dt in (F32, BF16):
        d_in, wr = torch.randn(T, E, generator=g), torch.randn(E, H, generator=g)
        x = torch.randn(T, H, generator=g).to(dt)
        d_in[3, 5], d_in[17, 2] = float("inf"), float("nan")
        wr[4, 9] = float("inf")
        x[20, 30] = float("nan")
        ids, w = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
        d_x = torch.empty(T, H, dtype=dt, device=DEV)
        d_wr, d_b = torch.empty(E, H, device=DEV), torch.empty(E, device=DEV)
        moe.moe_route_backward(x.to(DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), None, d_in.to(DEV),
                               torch.empty(T, E, device=DEV), d_x=d_x, d_w_router=d_wr, d_bias=d_b)
        bad = ~torch.isfinite(d_x.float()).cpu()
        assert bad[3].all() and bad[17].all() and bad[:, 9].all()
        keep = torch.ones(T, H, dtype=torch.bool)
        keep[3], keep[17], keep[:, 9] = False, False, False
        assert not bad[keep].any()
        bad = ~torch.isfinite(d_wr).cpu()
        assert bad[5].all() and bad[2].all() and bad[:, 30].all()
        keep = torch.ones(E, H, dtype=torch.bool)
        keep[5], keep[2], keep[:, 30] = False, False, False
        assert not bad[keep].any()
        assert torch.isfinite(d_b).cpu().nonzero().numel() == E - 2


def test_route_backward_repeated_and_outside_ids():
    g = torch.Generator().manual_seed(6)
    T, H, E, k = 20, 64, 8, 3
    x, wr = torch.randn(T, H, generator=g), torch.randn(E, H, generator=g)
    ids = torch.randint(0, E, (T, k), generator=g).int()
    ids[3], ids[4, 1], ids[5, 2] = 2, -1, E
    w, d_w = torch.rand(T, k, generator=g), torch.randn(T, k, generator=g)
    dl = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(x.to(DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), d_w.to(DEV), None, dl)
    ref, bound = route_backward(x.double(), wr.double(), ids.long(), w.double(), d_w.double(), None, False)["d_logits"]
    assert within(dl.cpu(), ref, bound, F32) <= 1.0


def test_route_backward_without_tokens():
    d_wr, d_b = torch.full((8, 64), -9.0, device=DEV), torch.full((8,), -9.0, device=DEV)
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device=DEV)
    moe.moe_route_backward(e(0, 64, dt=BF16), torch.ones(8, 64, device=DEV), e(0, 2, dt=torch.int32), e(0, 2), e(0, 2), None,
                           e(0, 8), d_x=e(0, 64, dt=BF16), d_w_router=d_wr, d_bias=d_b)
    assert not d_wr.any() and not d_b.any()


def test_int8_experts_and_the_router_tuned_to_them():
    """route -> balance loss -> int8 dispatch, experts, combine -> gradients of a loss on y and of the balance loss with
    respect to the router: eager, on a side stream and in a replayed graph. The gradients against float64 autograd through the
    softmax, the kernel's own expert outputs and the balance loss."""
    g = torch.Generator().manual_seed(12)
    T, H, E, k, F, C = 90, 64, 8, 2, 48, 30
    x = torch.randn(T, H, generator=g).to(BF16)
    wr, bias = torch.randn(E, H, generator=g) * 0.2, torch.randn(E, generator=g) * 0.1
    target = torch.randn(T, H, generator=g).to(BF16)
    dev = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device=DEV)
    gu, dn = torch.randn(E, 2 * F, H, generator=g) * 0.2, torch.randn(E, H, F, generator=g) * 0.2
    packs = []
    for w in (gu, dn):
        q, s = dev(*w.shape, dt=torch.int8), dev(*w.shape[:2])
        moe.moe_quantize_i8(w.to(DEV), q, s)
        packs += [q, s]
    xd, wrd, bd, td = x.to(DEV), wr.to(DEV), bias.to(DEV), target.to(DEV)
    logits, ids, w = dev(T, E), dev(T, k, dt=torch.int32), dev(T, k)
    L = moe.Layout(T, k, E, 1, C, H, device=DEV)
    sq, ss, out = dev(L.rows_max, H, dt=torch.int8), dev(L.rows_max), dev(L.rows_max, H, dt=BF16)
    y, dy = dev(T, H, dt=BF16), dev(T, H, dt=BF16)
    loss, count, d_bal, d_w = dev(1), dev(1, E, dt=torch.int32), dev(T, E), dev(T, k)
    d_x, d_wr, d_b = dev(T, H, dt=BF16), dev(E, H), dev(E)

    def step(**kw):
        moe.moe_route(xd, wrd, bd, k, logits, ids, w, **kw)
        moe.moe_balance_loss(logits, ids, 0.5, loss, count, d_logits=d_bal, **kw)
        moe.moe_dispatch_i8(xd, ids, L, sq, ss, **kw)
        moe.moe_expert_mlp_i8(sq, ss, L, *packs, out, **kw)
        moe.moe_combine(out, L, w, y, **kw)

    def back(**kw):
        moe.moe_combine_backward(dy, out, L, w, d_w, **kw)
        moe.moe_route_backward(xd, wrd, ids, w, d_w, d_bal, d_bal, d_x=d_x, d_w_router=d_wr, d_bias=d_b, **kw)

    step()
    dy.copy_(y - td)
    back()
    torch.cuda.synchronize()
    results = [t.clone() for t in (loss, count, y, d_w, d_bal, d_x, d_wr, d_b)]
    # autograd in float64 with the kernel's expert rows as constants
    w64, b64 = wr.double().requires_grad_(), bias.double().requires_grad_()
    x64 = x.double().requires_grad_()
    lg = x64 @ w64.T + b64
    sel = ids.cpu().long()
    p = torch.softmax(torch.gather(lg, 1, sel), 1)
    row = L.pair_row.cpu().long()
    o = out.cpu().double()
    yy = sum(torch.where(row[:, j:j + 1] >= 0, p[:, j:j + 1] * o[row[:, j].clamp(min=0)], torch.zeros(T, H).double())
             for j in range(k))
    f = count.cpu().double()[0] / (k * T)
    total = 0.5 * E * (f * torch.softmax(lg, 1).mean(0)).sum() + (yy * dy.cpu().double()).sum()
    total.backward()
    assert abs(float(loss) - float(0.5 * E * (f * torch.softmax(lg.detach(), 1).mean(0)).sum())) < 1e-5
    # the kernels' logits and weights are float32: off by some H 2^-24 of their terms' size, d_x also by bf16's half step
    for got, ref, rel in ((d_wr, w64.grad, 2e-5), (d_b, b64.grad, 2e-5), (d_x, x64.grad, 2.0 ** -8 + 2e-5)):
        assert float((got.cpu().double() - ref).norm() / ref.norm()) < rel

    def same():
        for a, b in zip((loss, count, y, d_w, d_bal, d_x, d_wr, d_b), results):
            assert torch.equal(a, b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    back(stream=side)
    torch.cuda.synchronize()
    same()
    with torch.cuda.stream(side):
        step()
        back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        back()
    for _ in range(3):
        for t in (loss, y, d_w, d_bal, d_x, d_wr, d_b, out):
            t.fill_(-3.0)
        graph.replay()
        torch.cuda.synchronize()
        same()
