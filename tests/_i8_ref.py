"""int8 rows and the int8 expert MLP in float64, with error bounds (U and silu's error: tests/_layer_ref.py).

The kernels' sums of int8 products are exact, so what is off is: g and u by three float32 roundings (the sum to float32, two
scales); h as in _layer_ref; the row's scale by h's error at its maximum and a division; a code by one step where 127 h / a
lies within h's error of a tie; the output by the sum to float32, two scales and the rounding to bf16, counted by `within`.
"""
from fractions import Fraction

import torch

from tests._layer_ref import SILU_REL, U


def levels(v):
    """float64 v [N, K] whose values are float32 -> (levels [N, K] float64, maxima [N]): 127 v is exact, and a quotient is
    rounded by its exact remainder."""
    top = v.abs().amax(1, keepdim=True)
    safe = torch.where(top == 0, torch.ones_like(top), top)
    # powers of two that keep tiny and huge rows' products in range
    unit = torch.exp2(torch.floor(torch.log2(safe)))
    v, safe = v / unit, safe / unit
    low = torch.floor(127.0 * v / safe)
    rest = 127.0 * v - low * safe
    up = (2 * rest > safe) | ((2 * rest == safe) & (low % 2 != 0))
    return low + up, top.squeeze(1)


def level_by_fractions(v, top):
    """One level from whole-number arithmetic."""
    if top == 0:
        return 0
    return round(Fraction(127) * Fraction(v) / Fraction(top))  # Python rounds halves to even


def expert(q, s, gu_q, gu_s, dn_q, dn_s):
    """(out, bound) of one expert for rows of codes q [n, H] with scales s [n]; all float64."""
    F = dn_q.shape[1]
    v = (q @ gu_q.T) * s.unsqueeze(1) * gu_s
    g, u = v[:, :F], v[:, F:]
    act = g / (1.0 + torch.exp(-g))
    h = act * u
    dh = (1.1 * 3 * U * g.abs() + SILU_REL * act.abs()) * u.abs() * (1 + 4 * U) + 4 * U * h.abs()
    a, at = h.abs().max(1, keepdim=True)
    safe = torch.where(a == 0, torch.ones_like(a), a)
    da = (dh + h.abs()).amax(1, keepdim=True) - a + dh.amax(1, keepdim=True)
    x = 127.0 * h / safe
    lv = torch.round(x)
    slack = 127.0 * (dh + h.abs() * da / safe) / safe
    may_flip = ((x - torch.floor(x) - 0.5).abs() <= slack).double()
    step = safe / 127.0
    out = (lv @ dn_q.T) * step * dn_s
    bound = out.abs() * (da / safe + 8 * U) + (may_flip @ dn_q.abs().T) * step * dn_s * (1 + 8 * U)
    return torch.where(a == 0, torch.zeros_like(out), out), torch.where(a == 0, torch.zeros_like(out), bound)
