"""4-bit weights: E2M1 codes with one E8M0 scale byte per 32 consecutive k, and their packed tile layout.

Test infrastructure (float64 numpy). The definitions are include/moe.h's, "4-bit expert weights": a code's value is
its magnitude (0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 the sign) times 2^(s - 127); E = s - 127 is the smallest integer with
max|w| <= 6 * 2^E over the group, clamped to [-120, 125], 0 for a group of zeros.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(w) -> tuple[np.ndarray, np.ndarray]:
    """w [N, K] float64 -> (codes [N, K] uint8 0..15, scale bytes [N, K / 32] uint8)."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((N, K // GROUP), np.uint8)
    # the value halfway between neighbouring magnitudes goes to the even code
    mid = (MAGNITUDES[:-1] + MAGNITUDES[1:]) / 2
    for n in range(N):
        for g in range(K // GROUP):
            v = w[n, g * GROUP:(g + 1) * GROUP]
            top = float(np.max(np.abs(v)))
            E = 0
            if top > 0:
                E = math.frexp(top)[1] - 4
                while 6.0 * math.ldexp(1.0, E) < top:
                    E += 1
                E = min(125, max(-120, E))
            scales[n, g] = E + 127
            q = np.abs(v) / math.ldexp(1.0, E)
            c = np.zeros(GROUP, np.uint8)
            for i, m in enumerate(mid):
                c += ((q > m) | ((q == m) & (i % 2 == 1))).astype(np.uint8)
            codes[n, g * GROUP:(g + 1) * GROUP] = c | (np.signbit(v).astype(np.uint8) << 3)
    return codes, scales


def values(codes, scales) -> np.ndarray:
    """The float64 values codes [N, K] and scale bytes [N, K / 32] stand for."""
    mag = MAGNITUDES[np.asarray(codes) & 7]
    sign = np.where(np.asarray(codes) & 8, -1.0, 1.0)
    return sign * mag * np.repeat(np.exp2(np.asarray(scales).astype(np.float64) - 127), GROUP, axis=1)


def pack(codes, scales) -> tuple[np.ndarray, np.ndarray]:
    """Codes [N, K], scale bytes [N, K / 32] -> tiles [N/16, ceil(K/128), 1024], [N/16, ceil(K/512), 256]."""
    N, K = codes.shape
    kc, ks = -(-K // 128), -(-K // 512)
    tc = np.zeros((N // 16, kc, 1024), np.uint8)
    ts = np.full((N // 16, ks, 256), 127, np.uint8)
    for n in range(N):
        for k in range(0, K, 2):
            lane = n % 16 + 16 * ((k % 128) // 32)
            tc[n // 16, k // 128, lane * 16 + (k % 32) // 2] = codes[n, k] | (codes[n, k + 1] << 4)
        for k in range(0, K, GROUP):
            lane = n % 16 + 16 * ((k % 128) // 32)
            ts[n // 16, k // 512, lane * 4 + (k % 512) // 128] = scales[n, k // GROUP]
    return tc, ts


def unpack(tc, ts, K) -> tuple[np.ndarray, np.ndarray]:
    """The inverse of pack for K columns."""
    nb, kc, ks = tc.shape[0], tc.shape[1], ts.shape[1]
    b = tc.reshape(nb, kc, 4, 16, 16).transpose(0, 3, 1, 2, 4).reshape(nb * 16, kc * 64)
    codes = np.stack([b & 15, b >> 4], axis=2).reshape(nb * 16, kc * 128)[:, :K]
    s = ts.reshape(nb, ks, 4, 16, 4).transpose(0, 3, 1, 4, 2).reshape(nb * 16, ks * 16)[:, :K // GROUP]
    return np.ascontiguousarray(codes), np.ascontiguousarray(s)
