"""The MoE layer and the expert MLP in float64 with error bounds, for the 4-bit and few-token tests.

Bounds are worst-case, from u = 2^-24 (half a step of float32, relative) for every float32 addition of exact
products: a sum of n products is off by at most (n + 1) u times the sum of their absolute values, in any order of
addition. silu and its division are off by at most 2^-20 relative (expf and the division take a few steps of
2^-23), and |silu'| < 1.1. h kept in bits with half step r is off by r |h| more.
"""
import torch

U = 2.0 ** -24
SILU_REL = 2.0 ** -20


def expert(rows, gate_up, down, h_half_step):
    """(out, bound) of one expert for rows [n, H]: gate_up [2F, H], down [H, F], all float64."""
    F = down.shape[1]
    H = rows.shape[1]
    s = rows @ gate_up.T
    ds = (H + 1) * U * (rows.abs() @ gate_up.abs().T)
    g, u, dg, du = s[:, :F], s[:, F:], ds[:, :F], ds[:, F:]
    act = g / (1.0 + torch.exp(-g))
    h = act * u
    dh = (1.1 * dg + SILU_REL * act.abs()) * (u.abs() + du) + act.abs() * du
    dh = dh + h_half_step * (h.abs() + dh)
    out = h @ down.T
    return out, dh @ down.abs().T + (F + 1) * U * ((h.abs() + dh) @ down.abs().T)


def layer(x, w_router, bias, k, R, C, ids, get_expert, h_half_step):
    """The layer of x [T, H] (float64) with the given selection ids [T, k]: dict of y, its bound before the last
    rounding, logits and their bound. get_expert(l) -> (gate_up, down) in float64."""
    T, H = x.shape
    E = w_router.shape[0]
    El = E // R
    logits = x @ w_router.T
    dl = (H + 2) * U * (x.abs() @ w_router.abs().T)
    if bias is not None:
        logits = logits + bias
        dl = dl + 2 * U * logits.abs()
    sel = torch.gather(logits, 1, ids)
    w = torch.softmax(sel, dim=1)
    # exp of a difference: its argument is off by twice the largest logit error and by the rounding of the
    # subtraction; a few steps more for expf, the sum and the division
    dmax = torch.gather(dl, 1, ids).amax(1, keepdim=True)
    spread = (sel - sel[:, :1]).abs().amax(1, keepdim=True)
    dw = w * (4 * dmax + 4 * U * spread + 64 * U)
    y = torch.zeros(T, H, dtype=torch.float64)
    dy = torch.zeros_like(y)
    seen = [0] * E
    mag = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            seen[e] += 1
            if seen[e] > C:
                continue
            out, do = expert(x[t:t + 1], *get_expert(e % El), h_half_step)
            y[t] += w[t, j] * out[0]
            dy[t] += (w[t, j] + dw[t, j]) * do[0] + dw[t, j] * out[0].abs()
            mag[t] += w[t, j] * (out[0].abs() + do[0])
    dy = dy + (k + 8) * U * mag
    return dict(y=y, dy=dy, logits=logits, dlogits=dl, w=w, dw=dw)


def within(got, ref, bound, dtype):
    """got (rounded once to dtype) against ref with `bound` before that rounding: the largest |error| / allowance."""
    half = torch.finfo(dtype).eps / 2
    allow = bound + half * (ref.abs() + bound) + torch.finfo(dtype).tiny
    return float(((got.double() - ref).abs() / allow).max()) if got.numel() else 0.0
