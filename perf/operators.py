"""Measured cases of the rotary and block-scaled-cache operators.

Four operators: the rotation of queries or keys (dattn_rope), the paged append that rotates on
the way (dattn_rope_append), and the decode and the prefill over the 8-bit pool with one
power-of-two scale per block of 16 tokens and KV head (KV_FP8_BLOCK). ``run`` computes a case in
elementary torch operations, or, where ``own`` is true, with the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
NAMES = ("rope", "append", "decode", "prefill")


def listed():
    return [
        # the queries of 16 requests in a decode step: latency counts
        _rope("rope-step", B=16, T=1, H=32, d=128, rot=128, far=40000),
        # the queries of a prompt of 16K tokens, out of a fused q, k, v projection
        _rope("rope-prompt", B=1, T=16384, H=32, d=128, rot=128, fused=True, far=0),
        # the gradient of the rotated half of the head, fp32, neighbouring channels paired
        _rope("rope-gradient", B=3, T=1021, H=16, d=64, rot=32, interleaved=True, inverse=True,
              f32=True, far=100000),
        # one token of one request into a bf16 pool: the smallest append
        _append("append-one", B=1, T=1, Hq=32, Hkv=8, d=128, P=16, fmt="bf16", ctx=700, far=0),
        # a decode step of 64 ragged requests into the block-scaled pool, with page statistics,
        # positions stretched by parts
        _append("append-step", B=64, T=1, Hq=32, Hkv=8, d=128, P=64, fmt="fp8-block", ctx=1500,
                stats=True, far=60000, factor=8.0),
        # a chunk of a long prompt into the block-scaled pool
        _append("append-chunk", B=2, T=4093, Hq=32, Hkv=8, d=128, P=16, fmt="fp8-block", ctx=900,
                far=0),
        # a short conversation: latency counts
        _decode("decode-short", B=2, T=1, Hq=32, Hkv=8, d=128, P=16, lo=130, hi=300),
        # the batch of 8 x 32K tokens with as many KV heads as query heads
        _decode("decode-32k", B=8, T=1, Hq=32, Hkv=32, d=128, P=16, lo=32768, hi=32768),
        # ragged requests, two new tokens each (a draft token is checked)
        _decode("decode-ragged", B=24, T=2, Hq=32, Hkv=8, d=128, P=64, lo=1000, hi=40000),
        # the tails of four short prompts, ragged, not on block boundaries
        _prefill("prefill-tails", B=4, Tq=75, Hq=8, Hkv=2, d=64, P=16, lo=90, hi=700),
        # a 4K chunk of a 32K prompt, causal
        _prefill("prefill-chunk", B=1, Tq=4096, Hq=32, Hkv=8, d=128, P=16, lo=32768, hi=32768),
        # the same heads block-sparse: half of them streaming, half keeping listed blocks
        _prefill("prefill-sparse", B=1, Tq=2048, Hq=32, Hkv=8, d=128, P=64, lo=16333, hi=16333,
                 sparse=True),
    ]


def _rope(name, **kw):
    base = dict(op="rope", interleaved=False, inverse=False, f32=False, fused=False, factor=1.0)
    return {**base, **kw, **({"name": name} if name else {})}


def _append(name, **kw):
    base = dict(op="append", interleaved=False, stats=False, factor=1.0, rot=kw["d"])
    return {**base, **kw, **({"name": name} if name else {})}


def _decode(name, **kw):
    return {"op": "decode", **kw, **({"name": name} if name else {})}


def _prefill(name, **kw):
    return {"op": "prefill", "sparse": False, **kw, **({"name": name} if name else {})}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(NAMES)
    d = rng.choice((64, 128))
    P = rng.choice((16, 32, 64, 128))
    Hkv = rng.choice((1, 2, 4, 8, 16, 32))
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 8) if g * Hkv <= 32])
    rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
    if rng.random() < 0.5:
        rot = d
    if op == "rope":
        B = _log(rng, 1, 64)
        H = rng.choice((1, 5, 8, 16, 32))
        T = _log(rng, 1, max(1, 16384 * 32 // (B * H) // 2))
        return _rope("", B=B, T=T, H=H, d=d, rot=rot, interleaved=rng.random() < 0.5,
                     inverse=rng.random() < 0.5, f32=rng.random() < 0.3,
                     fused=rng.random() < 0.5, factor=rng.choice((1.0, 4.0, 32.0)),
                     far=rng.choice((0, 100000, 1000000)))
    if op == "append":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 8000 // B))
        return _append("", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, P=P, rot=rot,
                       fmt=rng.choice(("bf16", "fp8", "fp8-block", "fp8-block")),
                       ctx=_log(rng, 16, 1500), interleaved=rng.random() < 0.5,
                       stats=rng.random() < 0.5, factor=rng.choice((1.0, 8.0)),
                       far=rng.choice((0, 1000000)))
    if op == "decode":
        B = _log(rng, 1, 48)
        T = rng.choice([t for t in (1, 1, 2, 3, 4) if t * (Hq // Hkv) <= 8])
        hi = _log(rng, 64, max(65, min(131072, 4_000_000 // (B * Hkv))))
        return _decode("", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, P=P, lo=max(T, hi // 16), hi=hi)
    B = _log(rng, 1, 4)
    Tq = _log(rng, 1, 2048 // B)
    hi = _log(rng, Tq, 8192)
    return _prefill("", B=B, Tq=Tq, Hq=Hq, Hkv=Hkv, d=d, P=P, lo=max(Tq, hi // 3), hi=hi,
                    sparse=rng.random() < 0.4)


# ------------------------------------------------------------------------------- inputs

def _all_lens(c):
    """Lengths spread evenly over the logarithm of [lo, hi]."""
    u = (torch.arange(c["B"], dtype=torch.float64) + 0.5) / c["B"]
    L = torch.exp(math.log(c["lo"]) + u * (math.log(c["hi"]) - math.log(c["lo"])))
    return L.round().to(torch.int64).clamp(c["lo"], c["hi"])


def _lens(c, seed):
    """The lengths of the requests, in the seed's order."""
    return _all_lens(c)[torch.randperm(c["B"], generator=torch.Generator().manual_seed(seed))]


def _table(caps, seed, n=None):
    """Block table [B][max pages] over a shuffled pool; unmapped entries are -1."""
    n = n or int(caps.sum())
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed * 7 + 2))
    perm = perm[:int(caps.sum())]
    at = torch.arange(int(caps.max()))
    used = at[None, :] < caps[:, None]
    bt = torch.full((len(caps), len(at)), -1, dtype=torch.int32)
    bt[used] = perm.to(torch.int32)
    return bt.to(DEV), n


def _frequencies(c):
    """Inverse frequencies of the rotated pairs in 64 bits; factor > 1 stretches the slow ones
    by parts (turns over an original length of 8192 below 1: divided, above 4: kept)."""
    n = c["rot"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if c["factor"] != 1.0:
        keep = ((8192.0 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f / c["factor"] * (1 - keep) + f * keep
    return f


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (0 for 0)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def _block_pool(n, Hkv, P, d, gen):
    """A block-scaled pool of normal values: codes [n][Hkv][P][d] and scales, both of K or V."""
    x = torch.randn(n, Hkv, P // 16, 16, d, device=DEV, generator=gen).to(torch.bfloat16).float()
    s = _pow2_scale(x.abs().amax((3, 4)))
    codes = (x / s[..., None, None]).to(torch.float8_e4m3fn)
    return codes.view(n, Hkv, P, d), s


def _pool(c, n, gen):
    """Block-scaled pools of n pages and their scales."""
    kp, ks = _block_pool(n, c["Hkv"], c["P"], c["d"], gen)
    vp, vs = _block_pool(n, c["Hkv"], c["P"], c["d"], gen)
    flat = torch.zeros(-(-n * c["Hkv"] * (c["P"] // 16) // 2) * 4, device=DEV)
    flat[:2 * ks.numel()] = torch.stack((ks, vs), -1).reshape(-1)
    return {"k_pool": kp, "v_pool": vp, "kv_scale": flat}


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 7 + 3)
    s = {"case": c}
    if c["op"] == "rope":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        width = 3 * c["H"] if c["fused"] else c["H"]
        x = torch.randn(c["B"], c["T"], width, c["d"], device=DEV, generator=gen).to(dt)
        s["x"] = x[:, :, :c["H"]]
        start = torch.randint(0, c["far"] + 1, (c["B"], 1), device=DEV, generator=gen)
        s["positions"] = (start + torch.arange(c["T"], device=DEV)).to(torch.int32)
        s["out"] = torch.empty(c["B"], c["T"], c["H"], c["d"], dtype=dt, device=DEV)
    elif c["op"] == "append":
        _prepare_append(c, seed, gen, s)
    else:
        T = c["T"] if c["op"] == "decode" else c["Tq"]
        lens = _lens(c, seed)
        s["block_table"], n = _table((lens + c["P"] - 1) // c["P"], seed)
        s.update(_pool(c, n, gen))
        s["seq_lens"] = lens.to(torch.int32).to(DEV)
        shape = (c["B"], T, c["Hq"], c["d"])
        s["q"] = torch.randn(shape, device=DEV, generator=gen).to(torch.bfloat16)
        s["out"] = torch.empty(shape, device=DEV)
        s["scale"] = c["d"] ** -0.5
        if c["op"] == "prefill" and c["sparse"]:
            _prepare_sparse(c, lens, gen, s)
    if "rot" in c:
        s["inv_freq"] = _frequencies(c)
    if own:
        _prepare_own(c, s)
    return s


def _prepare_append(c, seed, gen, s):
    """A pool whose requests hold up to ctx tokens, and T new tokens out of a fused projection."""
    B, T, Hq, Hkv, d, P = (c[k] for k in ("B", "T", "Hq", "Hkv", "d", "P"))
    lens = torch.randint(0, c["ctx"] + 1, (B,),
                         generator=torch.Generator().manual_seed(seed * 7 + 4))
    bt, n = _table((lens + T + 31) // P + 1, seed, B * ((c["ctx"] + T + 31) // P + 1))
    s["block_table"], s["seq_lens"] = bt, lens.to(torch.int32).to(DEV)
    qkv = torch.randn(B, T, Hq + 2 * Hkv, d, device=DEV, generator=gen).to(torch.bfloat16)
    s["q"], s["k_new"], s["v_new"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    s["q_out"] = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device=DEV)
    s["kv_scale"] = None
    if c["fmt"] == "bf16":
        s["k_pool"], s["v_pool"] = (
            torch.randn(n, Hkv, P, d, device=DEV, generator=gen).to(torch.bfloat16)
            for _ in range(2))
    elif c["fmt"] == "fp8":
        x = torch.randn(2, n, Hkv, P, d, device=DEV, generator=gen)
        sc = x.abs().amax(-1) / 448.0
        s["k_pool"], s["v_pool"] = (x / sc[..., None]).to(torch.float8_e4m3fn).unbind(0)
        s["kv_scale"] = sc.view(2, n, Hkv, P // 16, 16).permute(1, 2, 3, 0, 4).contiguous()
    else:
        s.update(_pool(c, n, gen))
    s["stats"] = None
    if c["stats"]:
        st = torch.randn(n, Hkv, P // 16, 2, d, device=DEV, generator=gen).to(torch.bfloat16)
        s["stats"] = torch.stack((st.amax(3), st.amin(3)), 3)
    base = s["seq_lens"].to(torch.int64)[:, None]
    if c["far"]:  # positions other than the slots': tokens dropped from a longer stream
        base = base + torch.randint(0, c["far"] + 1, (B, 1), device=DEV, generator=gen)
    s["positions"] = (base + torch.arange(T, device=DEV)).to(torch.int32)


def _prepare_sparse(c, lens, gen, s):
    """Half of the KV heads stream (1 + 4 blocks), half keep 65% of the earlier blocks."""
    nb = -(-int(lens.max()) // 64)
    kinds = [1] * (c["Hkv"] // 2) + [2] * (c["Hkv"] - c["Hkv"] // 2)
    s["head_kind"] = torch.tensor(kinds, dtype=torch.int8, device=DEV)
    s["sink_blocks"], s["local_blocks"] = 1, 4
    at = torch.arange(nb, device=DEV)
    keep = torch.rand(c["B"], c["Hkv"], nb, nb, device=DEV, generator=gen) < 0.65
    keep = (keep & (at[None, :] < at[:, None])) | (at[None, :] == at[:, None])
    # ascending lists padded with -1
    order = torch.where(keep, at, nb).sort(-1).values
    s["block_lists"] = torch.where(order < nb, order, -1).to(torch.int32)


def _prepare_own(c, s):
    """The handles a program keeps: the rotation, the layout, the workspace."""
    import split_kv_decode_distattention_gb300 as dattn
    if "rot" in c:
        s["rotation"] = dattn.Rotation(c["rot"], interleaved=c["interleaved"],
                                       inv_freq=s["inv_freq"].tolist())
    if c["op"] == "rope":
        return
    fmt = {"bf16": dattn.KV_BF16, "fp8": dattn.KV_FP8_E4M3,
           "fp8-block": dattn.KV_FP8_BLOCK}[c.get("fmt", "fp8-block")]
    s["layout"] = dattn.KVLayout(s["k_pool"].shape[0], c["Hkv"], c["d"], c["P"],
                                 s["block_table"], fmt, s["kv_scale"])
    if c["op"] == "decode":
        s["ws"] = dattn.Workspace(c["B"], c["Hq"] * c["T"], c["Hkv"], c["d"])
    if c["op"] == "prefill":
        s["sparse"] = dattn.PrefillSparseConfig(
            s["head_kind"], s["sink_blocks"], s["local_blocks"],
            s["block_lists"]) if c["sparse"] else None


# ------------------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_attention,
            "prefill": _plain_attention}[c["op"]](c, state)


def _run_own(c, s):
    import split_kv_decode_distattention_gb300 as dattn
    if c["op"] == "rope":
        dattn.dattn_rope(s["rotation"], s["x"], s["out"], s["positions"], inverse=c["inverse"])
        return s["out"]
    if c["op"] == "append":
        # the lengths stay: the layers of a model share them, and the last one advances them
        dattn.dattn_rope_append(s["layout"], s["k_pool"], s["v_pool"], s["stats"], s["rotation"],
                                s["q"], s["k_new"], s["v_new"], s["q_out"], s["seq_lens"],
                                positions=s["positions"], advance=False)
        return _append_outputs(s, s["q_out"])
    if c["op"] == "decode":
        if c["T"] == 1:
            dattn.dattn_decode(s["layout"], s["k_pool"], s["v_pool"], s["q"][:, 0], s["scale"],
                               s["seq_lens"], s["out"], s["ws"])
        else:
            dattn.dattn_decode_multi(s["layout"], s["k_pool"], s["v_pool"], s["q"], s["scale"],
                                     s["seq_lens"], s["out"], s["ws"])
        return s["out"]
    dattn.dattn_prefill(s["layout"], s["k_pool"], s["v_pool"], s["q"], s["scale"], s["seq_lens"],
                        s["out"], sparse=s["sparse"])
    return s["out"]


def _append_outputs(s, q):
    """The rotated queries and the pool: its values, or its codes' values beside their scales."""
    out = {"q": q, "k": s["k_pool"], "v": s["v_pool"]}
    if s["kv_scale"] is not None:
        out["scale"] = s["kv_scale"]
    if s["stats"] is not None:
        out["stats"] = s["stats"]
    return out


def _rotate(c, x, positions, inv_freq, inverse):
    """x [B][T][H][d] fp32 rotated at positions [B][T]; angles in 64 bits."""
    ang = positions.double()[..., None] * inv_freq.to(x.device)
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    if inverse:
        sin = -sin
    r, n = c["rot"], c["rot"] // 2
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :n], x[..., n:r]
        y[..., :n], y[..., n:r] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(c, s):
    x = s["x"]
    return _rotate(c, x.float(), s["positions"], s["inv_freq"], c["inverse"]).to(x.dtype)


def _plain_append(c, s):
    P, T, d = c["P"], c["T"], c["d"]
    q = _rotate(c, s["q"].float(), s["positions"], s["inv_freq"], False).to(torch.bfloat16)
    k = _rotate(c, s["k_new"].float(), s["positions"], s["inv_freq"], False).to(torch.bfloat16)
    v = s["v_new"]
    # the new tokens by 16-token blocks of their requests: block j of request b starts at
    # base + 16 j, and new[b, j, i] tells which of its tokens come with this call
    start = s["seq_lens"].long()
    base = start // 16 * 16
    nb = (T + 30) // 16
    t = base[:, None, None] + 16 * torch.arange(nb, device=DEV)[:, None] + torch.arange(
        16, device=DEV)
    i = t - start[:, None, None]
    new = ((i >= 0) & (i < T))[:, :, None, :, None]
    old = (i < 0)[:, :, None, :, None]  # earlier tokens of the block
    i = i.clamp(0, T - 1)
    row = torch.arange(c["B"], device=DEV)[:, None, None]
    kb, vb = k[row, i].transpose(2, 3), v[row, i].transpose(2, 3)  # [B][nb][Hkv][16][d]
    page = s["block_table"].long()[row[..., 0], t[..., 0] // P]
    lp = t[..., 0] % P // 16
    lpv = (-1, c["Hkv"], P // 16, 16, d)
    if s["kv_scale"] is None:
        for pool, x in ((s["k_pool"], kb), (s["v_pool"], vb)):
            p = pool.view(lpv)
            p[page, :, lp] = torch.where(new, x, p[page, :, lp])
    elif c["fmt"] == "fp8":
        sc = s["kv_scale"]
        for at, (pool, x) in enumerate(((s["k_pool"], kb), (s["v_pool"], vb))):
            p = pool.view(torch.uint8).view(lpv)
            x = x.float()
            xs = x.abs().amax(-1) / 448.0
            code = (x / xs.clamp_min(1e-38)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            p[page, :, lp] = torch.where(new, code, p[page, :, lp])
            sc[page, :, lp, at] = torch.where(new[..., 0], xs, sc[page, :, lp, at])
    else:
        n = s["k_pool"].shape[0]
        sc = s["kv_scale"][:n * c["Hkv"] * (P // 16) * 2].view(n, c["Hkv"], P // 16, 2)
        for at, (pool, x) in enumerate(((s["k_pool"], kb), (s["v_pool"], vb))):
            p = pool.view(torch.uint8).view(lpv)
            x = torch.where(new, x.float(), 0.0)
            was, was_s = p[page, :, lp], sc[page, :, lp, at]
            now_s = _pow2_scale(x.abs().amax((3, 4)))
            any_old, any_new = old[:, :, :, 0, 0], new.any(3)[..., 0]
            now_s = torch.where(any_old, torch.maximum(was_s, now_s), now_s)
            now_s = torch.where(any_new, now_s, was_s)
            div = torch.where(now_s > 0, now_s, 1.0)[..., None, None]
            code = (x / div).to(torch.float8_e4m3fn).view(torch.uint8)
            moved = (was.view(torch.float8_e4m3fn).float() * (was_s[..., None, None] / div)).to(
                torch.float8_e4m3fn).view(torch.uint8)
            p[page, :, lp] = torch.where(new, code, torch.where(old & any_new[..., None, None],
                                                                moved, was))
            sc[page, :, lp, at] = now_s
    if s["stats"] is not None:
        st = s["stats"]
        was = st[page, :, lp]
        hi = torch.where(new, kb.float(), -math.inf).amax(3)
        lo = torch.where(new, kb.float(), math.inf).amin(3)
        o = old.any(3)
        hi = torch.where(o, torch.maximum(hi, was[..., 0, :].float()), hi)
        lo = torch.where(o, torch.minimum(lo, was[..., 1, :].float()), lo)
        now = torch.stack((hi, lo), -2).to(torch.bfloat16)
        st[page, :, lp] = torch.where(new.any(3)[..., None], now, was)
    return _append_outputs(s, q)


def _gathered(c, s, pool, at, dtype=torch.float32):
    """K or V of every request by token: [B][Hkv][tokens][d]."""
    n, P, d = pool.shape[0], c["P"], c["d"]
    pages = s["block_table"].long().clamp_min(0)
    sc = s["kv_scale"][:n * c["Hkv"] * (P // 16) * 2].view(n, c["Hkv"], P // 16, 2)[pages][..., at]
    x = pool.view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(dtype)
    x = x.view(*pages.shape, c["Hkv"], P // 16, 16, d) * sc[..., None, None].to(dtype)
    return x.transpose(1, 2).reshape(c["B"], c["Hkv"], -1, d)


def _kept(c, s, n):
    """Which keys each query token may see: [B][Hkv or 1][T][n]."""
    T = c["T"] if c["op"] == "decode" else c["Tq"]
    key = torch.arange(n, device=DEV)
    pos = s["seq_lens"].long()[:, None] - T + torch.arange(T, device=DEV)  # [B][T]
    keep = (key <= pos[..., None])[:, None]
    if "block_lists" not in s:
        return keep
    nb = s["block_lists"].shape[2]
    kb, qb = key // 64, pos // 64
    stream = (kb < s["sink_blocks"]) | (kb > qb[..., None] - s["local_blocks"])
    lists = s["block_lists"].long()
    by_block = torch.zeros(*lists.shape[:3], nb + 1, dtype=torch.bool, device=DEV)
    by_block.scatter_(3, torch.where(lists >= 0, lists, nb), True)
    at = torch.arange(c["B"], device=DEV)[:, None]
    chosen = by_block[at, :, qb].transpose(1, 2)  # [B][Hkv][T][blocks]
    chosen = chosen[..., kb.clamp_max(nb)]
    streaming = (s["head_kind"] == 2)[None, :, None, None]
    return keep & torch.where(streaming, stream[:, None], chosen)


def _plain_attention(c, s):
    B, T, Hq, d = s["q"].shape
    k, v = _gathered(c, s, s["k_pool"], 0), _gathered(c, s, s["v_pool"], 1)
    keep = _kept(c, s, k.shape[2])
    q = s["q"].float().view(B, T, c["Hkv"], -1, d).permute(0, 2, 3, 1, 4)  # [B][Hkv][g][T][d]
    x = torch.matmul(q.reshape(B, c["Hkv"], -1, d), k.transpose(2, 3)) * s["scale"]
    x = x.view(B, c["Hkv"], -1, T, k.shape[2])
    x = x.masked_fill_(~keep[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    e = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, c["Hkv"], -1, k.shape[2]), v).view(B, c["Hkv"], -1, T, d)
    o = o / torch.where(e > 0, e, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d)


# ------------------------------------------------------------------------------- accounting

def _seen(c, L):
    """Keys that the T query tokens of requests of lengths L see, a KV head's mean."""
    T = c["T"] if c["op"] == "decode" else c["Tq"]
    dense = (T * (L - T) + T * (T + 1) // 2).double()
    if not c.get("sparse"):
        return dense
    stream = T * L.clamp_max(5 * 64).double()
    half = c["Hkv"] // 2
    return (0.65 * dense * half + stream * (c["Hkv"] - half)) / c["Hkv"]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["T"] * c["H"]
        return {"bytes": n * c["d"] * 2 * (4 if c["f32"] else 2) + c["B"] * c["T"] * 4,
                "flops": 3 * n * c["rot"]}
    if c["op"] == "append":
        n, d = c["B"] * c["T"], c["d"]
        size = 2 if c["fmt"] == "bf16" else 1
        moved = c["Hq"] * d * 4 + c["Hkv"] * d * 2 * (2 + size)
        return {"bytes": n * (moved + 4), "flops": 3 * n * (c["Hq"] + c["Hkv"]) * c["rot"]}
    L = _all_lens(c)
    T = c["T"] if c["op"] == "decode" else c["Tq"]
    kv = c["Hkv"] * int(L.sum()) * (2 * c["d"] + 0.5)
    return {"bytes": kv + c["B"] * T * c["Hq"] * c["d"] * 6,
            "flops": 4 * c["Hq"] * c["d"] * float(_seen(c, L).sum())}


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _turn64(c, s["x"], s, -1.0 if c["inverse"] else 1.0)
    if c["op"] == "append":
        # the pool's new rows are rounded to their format: they have no value in 64 bits
        out = {"q": _turn64(c, s["q"], s, 1.0), "k": None, "v": None}
        if s["kv_scale"] is not None:
            out["scale"] = None
        if s["stats"] is not None:
            out["stats"] = None
        return out
    T, g = s["q"].shape[1], c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    n = s["k_pool"].shape[0] * c["Hkv"] * (c["P"] // 16)
    scale = s["kv_scale"][:2 * n].view(-1, c["Hkv"], c["P"] // 16, 2).double()
    for b in range(c["B"]):
        L = int(s["seq_lens"][b])
        pages = s["block_table"][b, :-(-L // c["P"])].long()
        pos = torch.arange(L - T, L, device=DEV)[:, None]
        for h in range(c["Hkv"]):
            kv = [(p.view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double()
                   * scale[pages, h, :, i].repeat_interleave(16, 1)[..., None]).flatten(0, 1)[:L]
                  for i, p in enumerate((s["k_pool"], s["v_pool"]))]
            keys = torch.arange(L, device=DEV)[None]
            see = keys <= pos
            if "block_lists" in s:
                if int(s["head_kind"][h]) == 2:
                    see &= (keys // 64 < 1) | (pos // 64 - keys // 64 < 4)
                else:
                    rows = s["block_lists"][b, h]
                    held = (rows[:, :, None] == torch.arange(rows.shape[0], device=DEV)).any(1)
                    see &= held[pos // 64, keys // 64]
            for j in range(h * g, h * g + g):
                w = torch.where(see, s["q"][b, :, j].double() @ kv[0].T / math.sqrt(c["d"]),
                                -math.inf)
                out[b, :, j] = torch.nan_to_num(torch.softmax(w, -1), nan=0.0) @ kv[1]
    return out


def _turn64(c, x, s, sign):
    """The rotation as a product with e^(i angle), pairs as complex numbers."""
    x, r = x.double(), c["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       sign * s["positions"].double()[..., None] * s["inv_freq"].to(DEV))
    if c["interleaved"]:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous())
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())
    z = torch.view_as_real(z * turn[:, :, None])
    z = z.flatten(-2) if c["interleaved"] else torch.cat((z[..., 0], z[..., 1]), -1)
    return torch.cat((z, x[..., r:]), -1)
