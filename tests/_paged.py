"""Random paged pools of every format with their values in 64 bits, made on the CPU without the library.

Rows that no request holds are poison: NaN values, NaN codes or NaN scales. What reads beyond a request's
tokens shows it.
"""
from __future__ import annotations

import numpy as np
import torch

FORMATS = ("bf16", "fp8", "int4", "mixed", "fp8-block")
CODES = {"bf16": 0, "fp8": 1, "int4": 2, "mixed": 3, "fp8-block": 5}  # KV_*


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).float().to(torch.bfloat16)


class Paged:
    """K and V of requests of lens[b] tokens. `shared` lists (first request, end, tokens): the full
    pages of those first tokens are the first request's in all of [first, end)."""

    def __init__(self, fmt, lens, Hkv, d, P, seed, spare=2, shared=(), extra_cols=1, table=None):
        rng = np.random.default_rng(seed)
        self.fmt, self.Hkv, self.d, self.P, self.lens = fmt, Hkv, d, P, list(lens)
        B = len(self.lens)
        n = [-(-x // P) for x in self.lens]
        pages = sum(n) + spare
        if table is None:
            perm = rng.permutation(pages)
            table = np.full((B, max(n + [1]) + extra_cols), -1, np.int32)
            at = 0
            for b in range(B):
                table[b, :n[b]] = perm[at:at + n[b]]
                at += n[b]
            for lo, hi, tokens in shared:
                lead = max(range(lo, hi), key=lambda b: self.lens[b]) if hi > lo else 0
                for b in range(lo, hi):
                    k = min(tokens // P, n[b])
                    table[b, :k] = table[lead, :k]
        self.table, self.pages = table, pages
        # held[page][slot]: a token of a request
        held = np.zeros((pages, P), bool)
        for b in range(B):
            for j in range(n[b]):
                held[table[b, j], :min(P, self.lens[b] - j * P)] = True
        self.head4 = [fmt == "int4" or (fmt == "mixed" and h % 2 == 1) for h in range(Hkv)]
        self.k, self.k_pool, ks = self._one(rng, held)
        self.v, self.v_pool, vs = self._one(rng, held)
        self.kv_scale = None
        if fmt == "fp8-block":
            flat = np.zeros(-(-pages * Hkv * (P // 16) // 2) * 4, np.float32)
            flat[:2 * ks.size] = np.stack((ks, vs), -1).reshape(-1)
            self.kv_scale = torch.from_numpy(flat)
        elif fmt != "bf16":
            s = np.stack([x.reshape(pages, Hkv, P // 16, 16) for x in (ks, vs)], 3)
            self.kv_scale = torch.from_numpy(np.ascontiguousarray(s))

    def _one(self, rng, held):
        """(values [pages][Hkv][P][d] in 64 bits, the pool, scales [pages][Hkv][P or P/16])."""
        shape = (self.pages, self.Hkv, self.P, self.d)
        hold = np.broadcast_to(held[:, None, :, None], shape)
        if self.fmt == "bf16":
            x = bf16(rng.standard_normal(shape))
            x[~torch.from_numpy(hold.copy())] = float("nan")
            return x.double().numpy(), x, None
        code8 = rng.integers(0, 256, shape).astype(np.uint8)
        code8[(code8 & 0x7f) == 0x7f] = 0x30  # no NaN among the held codes
        x8 = torch.from_numpy(code8).view(torch.float8_e4m3fn).double().numpy()
        code4 = rng.integers(-7, 8, shape)
        four = np.array(self.head4)[None, :, None, None]
        x = np.where(four, code4.astype(np.float64), x8)
        top = np.where(four, 7.0, 448.0)[..., 0]
        if self.fmt == "fp8-block":
            s = 2.0 ** rng.integers(-9, -6, shape[:2] + (self.P // 16,))
            rows = np.repeat(s, 16, 2)
        else:
            s = rows = (rng.uniform(0.5, 3.0, shape[:3]) / top).astype(np.float32).astype(np.float64)
            s = np.where(held[:, None, :], s, np.nan)  # poison
        x = np.where(hold, x * rows[..., None], np.nan)
        code8[~hold] = 0x7f
        h4 = [h for h in range(self.Hkv) if self.head4[h]]
        h8 = [h for h in range(self.Hkv) if not self.head4[h]]
        packed = (code4 + 8).astype(np.uint8)
        packed = packed[..., 0::2] | (packed[..., 1::2] << 4)
        pool = np.concatenate((code8[:, h8].reshape(-1), packed[:, h4].reshape(-1)))
        return x, torch.from_numpy(pool), s.astype(np.float32)

    def rows(self, what, b, lo=0, hi=None):
        """Tokens [lo, hi) of request b, [n][Hkv][d] in 64 bits."""
        t = np.arange(lo, self.lens[b] if hi is None else hi)
        x = self.k if what == "k" else self.v
        return x[self.table[b][t // self.P], :, t % self.P]

    def layout(self, dattn, dev="cuda"):
        sc = None if self.kv_scale is None else self.kv_scale.to(dev)
        heads = [2 if x else 1 for x in self.head4] if self.fmt == "mixed" else None
        return dattn.KVLayout(self.pages, self.Hkv, self.d, self.P,
                              torch.from_numpy(self.table.copy()).to(dev), CODES[self.fmt], sc, heads)

    def pools(self, dev="cuda"):
        return self.k_pool.to(dev), self.v_pool.to(dev)


def weight_error(fmt):
    """The relative error of a softmax weight on its way into the second product: two bf16 terms, the
    first rounded or cut (2^-8), the second rounded (2^-9 of that), with 2^-20 for the exponential;
    two fp16 terms with the quantized pools (2^-22)."""
    return 2.0 ** -20 + (2.0 ** -17 if fmt == "bf16" else 2.0 ** -22)


def check(got, m, e, ref, bound, t, rm, re, what):
    """Rows got [n][d] (and m, e [n]) against ref; bf16 outputs add their rounding, half a step."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    g = got.double().cpu().numpy()
    lim = bound[:, None] + half * np.abs(ref) + 1e-30
    bad = ~(np.abs(g - ref) <= lim)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} elements out of tolerance, worst "
                           f"{np.nanmax(np.abs(g - ref) / lim):.3g} of it")
    if m is not None:
        m, e = m.double().cpu().numpy(), e.double().cpu().numpy()
        empty = ~np.isfinite(rm)
        assert (m[empty] == -np.inf).all() and (e[empty] == 0).all(), f"{what}: empty rows"
        m, e, rm, re, t = (np.broadcast_to(x, rm.shape)[~empty] for x in (m, e, rm, re, t))
        assert (np.abs(m - rm) <= t + 2.0 ** -22 * np.abs(rm)).all(), f"{what}: m"
        # e moves with m's error as well as with the weights'
        assert (np.abs(e - re) <= (4 * t + 2.0 ** -22 * np.abs(rm)) * re).all(), f"{what}: e"
