"""GPU: d_x of bf16 layers where the sum over the experts cancels. A softmax's gradient sums to 0 over the experts, so what the
router's rows share drops out of d_x by definition, and an operand kept in fewer bits than float32 would leave its rounding.

The bound: a scaled operand a is kept as two fp16 parts, hi + lo, off by at most 2^-22 |a| (half a step of fp16, 2^-11, twice),
and below fp16's normal range by 2^-39 of the largest value of its token or column (2^-25 of what is put at 2^14 or above). Of
the product's four parts lo * lo, at most 2^-22 |a b|, is left out. The 3 E products are exact in float32 (22 bits), and each of
their additions is off by at most U of the sum of their sizes."""
import pytest
import torch

import combine_router_gemm_amd as moe
from tests._layer_ref import U, within
from tests._router_ref import route_backward
from tests.test_gpu_router_training import DEV, F32, top_ids

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def tight(dl, db, wr):
    """Bound of d_x for float64 dl, off by db, and wr."""
    E = wr.shape[0]
    size = (dl.abs() + db) @ wr.abs()
    low = 2.0 ** -39
    sa, sb = low * (dl.abs() + db).amax(1, keepdim=True), low * wr.abs().amax(0, keepdim=True)
    return (((3 * E + 2) * U + 3.01 * 2.0 ** -22) * size + db @ wr.abs() +
            1.01 * (sa * wr.abs().sum(0) + sb * (dl.abs() + db).sum(1, keepdim=True)) + E * sa * sb)


def case(T, H, E, k, shared, seed):
    """A router whose rows are `shared` times a common row and their own; the softmax's and a balance loss's gradients."""
    g = torch.Generator().manual_seed(seed)
    wr = (torch.randn(E, H, generator=g) + shared * torch.randn(1, H, generator=g)) * 0.02
    lg = torch.randn(T, E, generator=g)
    ids = top_ids(lg, k)
    w = torch.softmax(torch.gather(lg, 1, ids.long()), 1)
    d_w = torch.randn(T, k, generator=g) * 0.1
    p = torch.softmax(lg.double(), 1)
    f = torch.rand(E, generator=g).double()
    d_in = (p * (f - (p * f).sum(1, keepdim=True)) * 0.3).float()
    return torch.randn(T, H, generator=g).to(BF16), wr, ids, w, d_w, d_in


# joint and separate launches, 32 and 64 tokens per wave, up to 256 experts and more
@pytest.mark.parametrize("shared", [0.0, 3.0, 30.0, 100.0])
@pytest.mark.parametrize("T,H,E,k", [(64, 128, 64, 2), (33, 264, 12, 8), (700, 1184, 256, 8), (600, 2048, 500, 3)])
def test_what_the_routers_rows_share_cancels(T, H, E, k, shared):
    print(f"\n[gpu] d_x of a shared row {T} {H} {E} {k} {shared}", flush=True)
    x, wr, ids, w, d_w, d_in = case(T, H, E, k, shared, T + E)
    for use_w, use_in in ((True, False), (False, True), (True, True)):
        d_x, d_wr = torch.empty(T, H, dtype=BF16, device=DEV), torch.empty(E, H, device=DEV)
        a, b = d_w if use_w else None, d_in if use_in else None
        args = [x.to(DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), None if a is None else a.to(DEV),
                None if b is None else b.to(DEV), torch.empty(T, E, device=DEV)]
        moe.moe_route_backward(*args, d_x=d_x, d_w_router=d_wr)
        r = route_backward(x.double(), wr.double(), ids.long(), w.double(), None if a is None else a.double(),
                           None if b is None else b.double(), True)
        (dl, db), ref = r["d_logits"], r["d_x"][0]
        assert within(d_x.cpu(), ref, tight(dl, db, wr.double()), BF16) <= 1.0
        alone = torch.empty_like(d_x)
        moe.moe_route_backward(*args, d_x=alone)
        assert torch.equal(alone, d_x)


def test_values_of_one_token_and_column_far_apart():
    """Each product is held to the sizes of its own token's and column's largest values."""
    g = torch.Generator().manual_seed(77)
    T, H, E = 150, 264, 24
    spread = lambda *s: torch.randn(*s, generator=g) * torch.exp2(torch.randint(-30, 20, s, generator=g).float())
    wr, d_in = spread(E, H), spread(T, E)
    d_x = torch.empty(T, H, dtype=BF16, device=DEV)
    ids, w = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
    moe.moe_route_backward(torch.zeros(T, H, dtype=BF16, device=DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), None,
                           d_in.to(DEV), torch.empty(T, E, device=DEV), d_x=d_x)
    dl = d_in.double()
    assert within(d_x.cpu(), dl @ wr.double(), tight(dl, torch.zeros_like(dl), wr.double()), BF16) <= 1.0


# two workgroups to a CU, one, two blocks of columns with 32 and with 64 tokens per wave; and the joint launch
@pytest.mark.parametrize("T,E,joint", [(70, 12, False), (300, 200, False), (70, 300, False), (600, 300, False), (70, 12, True),
                                       (300, 200, True), (70, 300, True)])
def test_an_infinity_gives_what_float32_gives(T, E, joint):
    """An infinite gradient or weight: infinities of the products' signs, NaN where they cancel or meet a zero, whatever the
    size of the token's and the column's other values; and nothing else."""
    print(f"\n[gpu] d_x with infinities {T} {E} {joint}", flush=True)
    g = torch.Generator().manual_seed(E)
    H = 136
    d_in, wr = torch.randn(T, E, generator=g), torch.randn(E, H, generator=g)
    inf = float("inf")
    d_in[3, 5], d_in[3, 7], d_in[3, 8] = inf, -1e6, 1e30
    d_in[9, 2], d_in[9, 4] = -inf, inf
    d_in[17, 2] = float("nan")
    d_in[40], d_in[40, 1] = 0.0, -inf
    wr[4, 9], wr[6, 9], wr[7, 9] = inf, 3e30, 1e-30
    wr[1, 20], wr[1, 21] = 0.0, 1e-38
    wr[2, 33] = -inf
    d_x = torch.empty(T, H, dtype=BF16, device=DEV)
    ids, w = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
    moe.moe_route_backward(torch.zeros(T, H, dtype=BF16, device=DEV), wr.to(DEV), ids.to(DEV), w.to(DEV), None,
                           d_in.to(DEV), torch.empty(T, E, device=DEV), d_x=d_x,
                           d_w_router=torch.empty(E, H, device=DEV) if joint else None)
    ref = d_in.double() @ wr.double()
    got = d_x.cpu().double()
    bad = ~torch.isfinite(ref)
    assert bad[[3, 9, 17, 40]].all() and bad[:, [9, 33]].all()
    same = torch.equal(torch.nan_to_num(got[bad], nan=5.0), torch.nan_to_num(ref[bad], nan=5.0))
    assert same  # (a failure would spell out the tensors)
    fin = lambda t: torch.where(torch.isfinite(t), t, torch.zeros_like(t))
    dl, wf = fin(d_in.double()), fin(wr.double())
    got, ref = torch.where(bad, torch.zeros_like(got), got), torch.where(bad, torch.zeros_like(ref), ref)
    assert within(got.to(BF16), ref, tight(dl, torch.zeros_like(dl), wf), BF16) <= 1.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H,E", [(40, 136, 12), (300, 264, 130)])
def test_d_w_router_at_the_ends_of_the_range(T, H, E, dtype):
    """Gradients of the logits up to the largest float32 (beyond the largest bf16, 3.39e38, too), and infinite ones: infinities of
    the products' signs and NaN where they cancel or meet a zero, as in float32; the rest to the bound of its sums."""
    print(f"\n[gpu] d_w_router at the ends {T} {H} {E} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T + E)
    d_in, x = torch.randn(T, E, generator=g), torch.randn(T, H, generator=g).to(dtype)
    x[5:8] *= 2.0 ** -10
    big = torch.finfo(F32).max
    d_in[5, 1], d_in[6, 2], d_in[7, 3] = big, -big, 3.3960e38
    inf = float("inf")
    d_in[9, 4], d_in[10, 5], d_in[11, 5], d_in[12, 6] = -inf, inf, -inf, float("nan")
    x[9, 3] = 0.0
    ids, w = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
    d_wr, d_b = torch.empty(E, H, device=DEV), torch.empty(E, device=DEV)
    moe.moe_route_backward(x.to(DEV), torch.zeros(E, H, device=DEV), ids.to(DEV), w.to(DEV), None, d_in.to(DEV),
                           torch.empty(T, E, device=DEV), d_w_router=d_wr, d_bias=d_b)
    ref = d_in.double().T @ x.double()
    got, bad = d_wr.cpu().double(), ~torch.isfinite(ref)
    assert bad[4:7].all() and bad.sum() == 3 * H
    same = torch.equal(torch.nan_to_num(got[bad], nan=5.0), torch.nan_to_num(ref[bad], nan=5.0))
    assert same
    bound = (T + 2) * U * (torch.nan_to_num(d_in.double(), posinf=0.0, neginf=0.0).abs().T @ x.double().abs())
    assert within(torch.where(bad, torch.zeros_like(got), got), torch.where(bad, torch.zeros_like(ref), ref), bound, F32) <= 1.0
