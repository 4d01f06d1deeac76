"""GPU: the router's training calls at sizes where a workgroup goes through several tiles of tokens, or a group of lanes takes
several tokens at once, and where the two products are launches of their own. Oracle and bounds: tests/_router_ref.py."""
import pytest
import torch

import combine_router_gemm_amd as moe
from tests._layer_ref import within
from tests._router_ref import route_backward
from tests.test_gpu_router_training import BF16, DEV, F32, check_balance, top_ids

pytestmark = pytest.mark.gpu


# a workgroup takes 256 or 512 tokens of 128 or 64 columns, and at most 512 workgroups divided over the columns are launched;
# the launches are joined where they need no more than 256 workgroups in all
@pytest.mark.parametrize("T,H,E,k,dtype", [(4600, 7168, 256, 8, BF16), (4600, 7168, 256, 8, F32), (2200, 20480, 512, 8, BF16),
                                           (2200, 20480, 512, 8, F32), (9001, 8192, 40, 4, BF16), (9001, 8192, 40, 4, F32),
                                           (250, 20480, 400, 8, BF16), (250, 20480, 400, 8, F32)])
def test_route_backward_of_many_tiles(T, H, E, k, dtype):
    print(f"\n[gpu] route backward {T} {H} {E} {k} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T + H + E)
    x = torch.randn(T, H, generator=g).to(dtype)
    wr = torch.randn(E, H, generator=g) * 0.05
    lg = torch.randn(T, E, generator=g)
    ids = top_ids(lg, k)
    w = torch.softmax(torch.gather(lg, 1, ids.long()), 1)
    d_w, d_in = torch.randn(T, k, generator=g), torch.randn(T, E, generator=g) * 0.1
    dev = [t.to(DEV) for t in (x, wr, ids, w, d_w, d_in)]
    got = dict(d_logits=torch.full((T, E), -9.0, device=DEV), d_x=torch.full((T, H), -9.0, dtype=dtype, device=DEV),
               d_w_router=torch.full((E, H), -9.0, device=DEV), d_bias=torch.full((E,), -9.0, device=DEV))
    moe.moe_route_backward(*dev, got["d_logits"], d_x=got["d_x"], d_w_router=got["d_w_router"], d_bias=got["d_bias"])
    # every token in a sample of columns, and every column in a sample of tokens: tiles' ends among both
    cols = torch.unique(torch.cat([torch.arange(0, 70), torch.arange(H - 70, H), torch.randint(0, H, (120,), generator=g)]))
    r = route_backward(x[:, cols].double(), wr[:, cols].double(), ids.long(), w.double(), d_w.double(), d_in.double(),
                       dtype is BF16)
    for name, pick in (("d_logits", got["d_logits"]), ("d_bias", got["d_bias"]), ("d_x", got["d_x"][:, cols.to(DEV)]),
                       ("d_w_router", got["d_w_router"][:, cols.to(DEV)])):
        assert within(pick.cpu(), *r[name], pick.dtype) <= 1.0, name
    rows = torch.unique(torch.cat([torch.arange(T - 90, T), torch.randint(0, T, (60,), generator=g)]))
    r = route_backward(x[rows].double(), wr.double(), ids[rows].long(), w[rows].double(), d_w[rows].double(),
                       d_in[rows].double(), dtype is BF16)
    assert within(got["d_x"][rows.to(DEV)].cpu(), *r["d_x"], dtype) <= 1.0


# 64 lanes per token: 16 tokens at once, and 32 or 64 in a round of four; 16 lanes: 64; 4 lanes: 256; more than 256 experts take
# two at once, and single logits (an E that is no multiple of 4) as well
@pytest.mark.parametrize("T,E,k,S", [(5000, 256, 8, 1), (5000, 256, 8, 5), (33000, 256, 2, 3), (9000, 512, 8, 1), (9000, 384, 4, 4),
                                     (17500, 24, 3, 1), (40000, 24, 2, 7), (70000, 12, 2, 1), (70000, 12, 2, 4),
                                     (9000, 130, 2, 2), (9001, 61, 2, 1), (20000, 15, 2, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_of_many_tokens(T, E, k, S, masked):
    print(f"\n[gpu] balance {T} {E} {k} {S} {masked}", flush=True)
    g = torch.Generator().manual_seed(T + E + S)
    logits = torch.randn(T, E, generator=g) * 2 - 0.5 * torch.arange(E).float() / E
    cuts = sorted(torch.randint(0, T, (S - 1,), generator=g).tolist())
    offset = None if S == 1 else [5] + [max(5, c) for c in cuts] + [T - 77]
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if masked else None
    check_balance(logits, top_ids(logits, k), 0.7, offset, mask)
