"""GPU: the balance loss where nearly even choices are counted beyond 2^24. f enters the gradient less its smallest value, so
that a difference of counts is what is rounded, not the counts: p is 1/2 everywhere here and the gradient of expert 0 is
weight * E / T * 1/2 * (c0 - c1) / (2 T), whose factors are powers of two but for the difference."""
import pytest
import torch

import combine_router_gemm_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("more", [1, 3, 1001])
@pytest.mark.parametrize("offset", [None, [0, 1 << 25], [0] * 12 + [1 << 25]])
def test_nearly_even_counts_keep_their_difference(more, offset):
    T = 1 << 25
    print(f"\n[gpu] balance {T} {more} {None if offset is None else len(offset) - 1}", flush=True)
    S = 1 if offset is None else len(offset) - 1
    logits = torch.zeros(T, 2, device=DEV)
    ids = torch.ones(T, 1, dtype=torch.int32, device=DEV)
    ids[:T // 2 + more] = 0
    loss, count = torch.empty(1, device=DEV), torch.empty(S, 2, dtype=torch.int32, device=DEV)
    d = torch.full((T, 2), -9.0, device=DEV)
    off = None if offset is None else torch.tensor(offset, dtype=torch.int32, device=DEV)
    moe.moe_balance_loss(logits, ids, 1.0, loss, count, d_logits=d, seq_offset=off)
    assert count[-1].tolist() == [T // 2 + more, T // 2 - more]
    want = 2.0 / T * 0.5 * (2 * more) / (2 * T)
    same = bool((d[:, 0] == want).all()) and bool((d[:, 1] == -want).all())
    assert same  # (a failure would spell out the tensors)
    assert abs(float(loss) - 1.0) <= 16 * 2.0 ** -24
