"""Plain 64-bit references of the rotation and of the block-scaled 8-bit pool, for the tests.

Nothing here calls the library. Angles are exact rational multiples of a turn until the final
sine and cosine; E4M3 rounding is torch's float8_e4m3fn conversion on the CPU, after clamping to
+-448 (the format's saturation).
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

# 2 pi to 60 digits
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194989")


def angles(positions, inv_freq):
    """[N][n] angles in [0, 2 pi), of the exact product reduced exactly."""
    turns = [Fraction(float(f)) / TWO_PI for f in inv_freq]
    out = np.empty((len(positions), len(turns)))
    for i, p in enumerate(positions):
        for k, t in enumerate(turns):
            out[i, k] = float((int(p) * t) % 1) * float(TWO_PI)
    return out


def rotate(x, positions, inv_freq, interleaved=False, inverse=False, amplitude=1.0):
    """x float64 [N][H][d] rotated at positions [N]; rot_dim = 2 len(inv_freq)."""
    x = np.asarray(x, np.float64)
    n = len(inv_freq)
    a = angles(positions, inv_freq)
    cos, sin = np.cos(a)[:, None] * amplitude, np.sin(a)[:, None] * amplitude
    if inverse:
        sin = -sin
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n),
                                                                          slice(n, 2 * n))
    y = x.copy()
    y[..., ia] = x[..., ia] * cos - x[..., ib] * sin
    y[..., ib] = x[..., ib] * cos + x[..., ia] * sin
    return y


def partner_sum(x, n, interleaved=False):
    """|x_a| + |x_b| of every channel's pair (0 for the unrotated channels)."""
    x = np.abs(np.asarray(x, np.float64))
    s = np.zeros_like(x)
    if interleaved:
        s[..., 0:2 * n:2] = s[..., 1:2 * n:2] = x[..., 0:2 * n:2] + x[..., 1:2 * n:2]
    else:
        s[..., :n] = s[..., n:2 * n] = x[..., :n] + x[..., n:2 * n]
    return s


def e4m3(x):
    """E4M3 codes (uint8) of float32 values, saturated."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).clamp(-448.0, 448.0)
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_values(codes):
    t = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn)
    return t.to(torch.float64).numpy()


def block_scale(m):
    """The smallest power of two s in [2^-126, 2^119] with m <= 448 s; 0 for 0."""
    if m == 0:
        return 0.0
    for k in range(-126, 120):
        if m <= 448.0 * 2.0 ** k:
            return 2.0 ** k
    return 2.0 ** 119


class BlockPool:
    """Codes [pages][Hkv][P][d] and scales [pages][Hkv][P/16] of K or of V."""

    def __init__(self, pages, Hkv, P, d, codes=0, scale=0.0):
        self.P = P
        self.codes = np.full((pages, Hkv, P, d), codes, np.uint8)
        self.scale = np.full((pages, Hkv, P // 16), scale, np.float32)

    def append(self, table, pos0, rows):
        """One call's rows [T][Hkv][d] (float) of one request at positions pos0 ..."""
        rows = np.asarray(rows, np.float64)
        T = rows.shape[0]
        for b0 in range(pos0 // 16 * 16, pos0 + T, 16):
            lo, hi = max(b0, pos0), min(b0 + 16, pos0 + T)
            page, lp = table[b0 // self.P], b0 % self.P // 16
            if page < 0 or page >= len(self.codes):
                continue
            s0 = b0 % self.P
            for h in range(rows.shape[1]):
                new = rows[lo - pos0:hi - pos0, h]
                s = block_scale(np.abs(new).max())
                was = float(self.scale[page, h, lp]) if lo > b0 else 0.0
                s = max(s, was)
                code = self.codes[page, h]
                if s > was > 0:
                    old = e4m3_values(code[s0:s0 + lo - b0])
                    code[s0:s0 + lo - b0] = e4m3((old * (was / s)).astype(np.float32))
                q = new / s if s > 0 else new * 0.0
                code[s0 + lo - b0:s0 + hi - b0] = e4m3(q.astype(np.float32))
                self.scale[page, h, lp] = s

    def values(self, table, L):
        """Token-ordered values [L][Hkv][d] of a request."""
        n = -(-L // self.P)
        pages = np.asarray(table[:n])
        v = e4m3_values(self.codes[pages]) * np.repeat(self.scale[pages].astype(np.float64), 16,
                                                      2)[..., None]
        return v.transpose(0, 2, 1, 3).reshape(n * self.P, *v.shape[1:2], v.shape[3])[:L]


def attention(q, K, V, scale, see=None, weights=2.0 ** -20):
    """float64 softmax attention of q [T][d] over K, V [L][d]; see [T][L] marks the visible keys.
    Returns out, m, e and an error bound of out for a computation whose logits are sums of d
    exact products in fp32 (in any order: d * 2^-23 of the sum of magnitudes, its scaling
    included), whose weights have a relative error `weights`, and whose weighted sums take in 16
    keys at a time in fp32 (2^-23 of the sum of magnitudes each time): a relative error t of the
    weights changes a weighted mean of values by at most 2 t max|v|. Also returns t."""
    q, K, V = (np.asarray(t, np.float64) for t in (q, K, V))
    s = q @ K.T * scale
    if see is not None:
        s = np.where(see, s, -np.inf)
    m = s.max(-1, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
    e = p.sum(-1)
    out = p @ V / np.where(e > 0, e, 1.0)[:, None]
    mag = np.abs(q) @ np.abs(K).T * abs(scale)
    if see is not None:
        mag = np.where(see, mag, 0.0)
    t = q.shape[1] * 2.0 ** -23 * mag.max(-1, initial=0.0) + weights + (
        K.shape[0] / 16 + 1) * 2.0 ** -23
    bound = 2.0 * t * (np.abs(V).max(initial=0.0))
    return out, m, e, bound, t
