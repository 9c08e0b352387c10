"""Measured cases of the shared-prefix decode, the sliding windows and the reading back of a cache.

Four operators over the paged cache: the decode of a batch whose requests share long prefixes
(dattn_decode_shared), the sliding window with first tokens that stay visible, in a prefill chunk
(dattn_prefill_window) and in a step of one or a few tokens (dattn_decode_window), and the cache's
rows read back out of pages and codes (dattn_kv_read). ``run`` computes a case in elementary torch
operations, or, where ``own`` is true, with the library's calls. The attention's outputs are bf16,
as the output projection takes them.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
NAMES = ("shared", "window", "step", "read")


def listed():
    return [
        # a few chats behind one system prompt, just begun: latency counts
        _shared("shared-few", sizes=4, prefix=1808, Hq=32, Hkv=8, d=128, P=16, lo=20, hi=90),
        # 64 questions about one long document
        _shared("shared-batch", sizes=64, prefix=16384, Hq=32, Hkv=8, d=128, P=64, lo=100, hi=2000),
        # three prompts of their own length with 32 requests behind them, a draft token checked,
        # 8-bit cache
        _shared("shared-block", sizes=32, groups=3, prefix=24576, T=2, Hq=32, Hkv=8, d=128, P=16,
                lo=50, hi=1500, fmt="fp8-block"),
        # the tails of five short prompts, on no block boundary, a window of no round size
        _window("window-tails", B=5, Tq=77, Hq=8, Hkv=2, d=64, P=16, lo=90, hi=900, W=333, S=4),
        # a whole prompt of 16K tokens through a window of 1024
        _window("window-prompt", B=1, Tq=16384, Hq=32, Hkv=8, d=128, P=64, lo=16384, hi=16384,
                W=1024, S=4),
        # a 4K chunk after 28K tokens through a window of 4096, 8-bit cache
        _window("window-chunk", B=1, Tq=4096, Hq=32, Hkv=8, d=128, P=16, lo=32768, hi=32768,
                W=4096, S=64, fmt="fp8-block"),
        # four draft tokens of two requests, a short window: latency counts
        _step("step-draft", B=2, T=4, Hq=16, Hkv=8, d=128, P=16, lo=200, hi=3000, W=512, S=4),
        # a ragged batch with a draft token each, row-scaled 8-bit cache
        _step("step-batch", B=64, T=2, Hq=32, Hkv=8, d=128, P=64, lo=1000, hi=40000, W=4096, S=16,
              fmt="fp8"),
        # one short request out of a 4-bit cache
        _read("read-one", B=1, Hkv=8, d=128, P=16, lo=300, hi=300, fmt="int4"),
        # eight requests leave an 8-bit cache for another instance
        _read("read-batch", B=8, Hkv=8, d=128, P=64, lo=4000, hi=12000, fmt="fp8-block"),
        # stretches in the middle of three requests, 8-bit and 4-bit heads, for a check in fp32
        _read("read-middle", B=3, Hkv=16, d=128, P=32, lo=1501, hi=6007, fmt="mixed", f32=True,
              middle=True),
    ]


def _named(name, c):
    return {**c, **({"name": name} if name else {})}


def _shared(name, **kw):
    return _named(name, {"op": "shared", "fmt": "bf16", "T": 1, "groups": 1, **kw})


def _window(name, **kw):
    return _named(name, {"op": "window", "fmt": "bf16", **kw})


def _step(name, **kw):
    return _named(name, {"op": "step", "fmt": "bf16", **kw})


def _read(name, **kw):
    return _named(name, {"op": "read", "f32": False, "middle": False, **kw})


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(NAMES)
    d = rng.choice((64, 128))
    P = rng.choice((16, 32, 64, 128))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    g = rng.choice([g for g in (1, 2, 3, 4, 8) if g * Hkv <= 32])
    T = rng.choice([t for t in (1, 1, 2, 3, 4) if t * g <= 8])
    heads = {"Hq": g * Hkv, "Hkv": Hkv, "d": d, "P": P}
    block = rng.choice(("bf16", "fp8-block"))
    if op == "shared":
        sizes = _log(rng, 2, 64)
        prefix = _log(rng, 128, min(32768, 1_000_000 // sizes, 131072 // Hkv))
        return _shared("", sizes=sizes, groups=rng.randint(1, min(4, sizes)), prefix=prefix, T=T,
                       lo=T, hi=T + _log(rng, 1, 1500), fmt=block, **heads)
    if op == "window":
        B = _log(rng, 1, 6)
        Tq = _log(rng, 1, 4096 // B)
        hi = Tq + _log(rng, 1, 12000)
        return _window("", B=B, Tq=Tq, lo=max(Tq, hi // 3), hi=hi, W=_log(rng, 1, 4096),
                       S=rng.choice((0, 1, 4, 64, 130)), fmt=block, **heads)
    fmt = rng.choice(("bf16", "fp8", "int4", "mixed", "fp8-block"))
    if op == "step":
        B = _log(rng, 1, 48)
        hi = _log(rng, 64, 400_000 // B)
        return _step("", B=B, T=T, lo=max(T, hi // 16), hi=hi, W=_log(rng, 1, 8192),
                     S=rng.choice((0, 1, 4, 64, 130)), fmt=fmt, **heads)
    B = _log(rng, 1, 32)
    hi = _log(rng, 8, 60000 // B)
    return _read("", B=B, Hkv=Hkv, d=d, P=P, lo=max(1, hi // 8), hi=hi, fmt=fmt,
                 f32=rng.random() < 0.3, middle=rng.random() < 0.4)


# ------------------------------------------------------------------------------- inputs

def _spread(lo, hi, n):
    """n lengths spread evenly over the logarithm of [lo, hi]."""
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    x = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))
    return x.round().to(torch.int64).clamp(lo, hi)


def _perm(n, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed))


def _sizes(c):
    """Requests of every group, and the groups' prefixes: from the listed one down to a sixth."""
    n, g = c["sizes"], c["groups"]
    at = (torch.arange(g + 1, dtype=torch.float64) / g) ** 1.5
    ends = (at * (n - g)).round().to(torch.int64) + torch.arange(g + 1)
    top = c["prefix"]
    return ends, _spread(max(1, top // 6), top, g).flip(0) if g > 1 else torch.tensor([top])


def _pages(c):
    """Pages of the pool: the requests' tokens, the groups' prefixes, and a few that nothing uses."""
    P = c["P"]
    n = c.get("B", c.get("sizes"))
    pages = int((_spread(c["lo"], c["hi"], n) // P).sum()) + 2 * n + 3
    return pages + (int((_sizes(c)[1] // P).sum()) if c["op"] == "shared" else 0)


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (0 for 0)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def _four(fmt, Hkv):
    """Which KV heads hold 4-bit codes."""
    return [fmt == "int4" or (fmt == "mixed" and h % 3 != 0) for h in range(Hkv)]


def _pool(c, n, gen):
    """K and V pools of n pages of normal values, and their scales."""
    Hkv, P, d, fmt = c["Hkv"], c["P"], c["d"], c["fmt"]
    if fmt == "bf16":
        return {"k_pool": torch.randn(n, Hkv, P, d, device=DEV, generator=gen).to(torch.bfloat16),
                "v_pool": torch.randn(n, Hkv, P, d, device=DEV, generator=gen).to(torch.bfloat16),
                "kv_scale": None}
    pools, scales = [], []
    four = _four(fmt, Hkv)
    h4 = torch.tensor([h for h in range(Hkv) if four[h]], dtype=torch.int64, device=DEV)
    h8 = torch.tensor([h for h in range(Hkv) if not four[h]], dtype=torch.int64, device=DEV)
    most = torch.where(torch.tensor(four, device=DEV), 7.0, 448.0)[:, None]
    for _ in range(2):
        x = torch.randn(n, Hkv, P, d, device=DEV, generator=gen)
        if fmt == "fp8-block":
            s = _pow2_scale(x.view(n, Hkv, P // 16, 16, d).abs().amax((3, 4)))
            pools.append((x / s.repeat_interleave(16, 2)[..., None]).to(torch.float8_e4m3fn)
                         .view(torch.uint8).view(-1))
        else:
            s = x.abs().amax(-1) / most
            x = x / s[..., None]
            e8 = x[:, h8].to(torch.float8_e4m3fn).view(torch.uint8)
            e4 = (x[:, h4].round().clamp(-7, 7) + 8).to(torch.uint8)
            e4 = e4[..., 0::2] | (e4[..., 1::2] << 4)
            pools.append(torch.cat((e8.reshape(-1), e4.reshape(-1))))
        scales.append(s)
    if fmt == "fp8-block":
        flat = torch.zeros(-(-n * Hkv * (P // 16) // 2) * 4, device=DEV)
        flat[:2 * scales[0].numel()] = torch.stack(scales, -1).reshape(-1)
    else:
        flat = torch.stack([s.view(n, Hkv, P // 16, 16) for s in scales], 3).reshape(-1)
    return {"k_pool": pools[0], "v_pool": pools[1], "kv_scale": flat}


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 7 + 3)
    s = {"case": c}
    B, P = c.get("B", c.get("sizes")), c["P"]
    lens = _spread(c["lo"], c["hi"], B)[_perm(B, seed)]
    if c["op"] == "shared":
        ends, prefix = _sizes(c)
        of = torch.repeat_interleave(torch.arange(c["groups"]), ends[1:] - ends[:-1])
        lens = lens + prefix[of]  # the prefix, then tokens of the request's own
        s["group_indptr"] = ends.to(torch.int32).to(DEV)
    caps = (lens + P - 1) // P
    at = torch.arange(int(caps.max()))
    used = at[None, :] < caps[:, None]
    if c["op"] == "shared":  # the prefix's full pages are the group's; a page begun in it is not
        first = ends[:-1][of]
        same = (at[None, :] + 1) * P <= prefix[of][:, None]
        used &= ~same | (first == torch.arange(B))[:, None]
        s["prefix_lens"] = (prefix // P * P).to(torch.int32).to(DEV)
    s["pages"] = _pages(c)
    table = torch.full(used.shape, -1, dtype=torch.int64)
    table[used] = _perm(s["pages"], seed * 7 + 2)[:int(used.sum())]
    if c["op"] == "shared":
        table = torch.where(same, table[first], table)
    s["block_table"] = table.to(torch.int32).to(DEV)
    s["seq_lens"] = lens.to(torch.int32).to(DEV)
    s.update(_pool(c, s["pages"], gen))
    if c["op"] == "read":
        count = lens
        if c["middle"]:  # the second and third quarter of each request
            count = (lens // 2).clamp_min(1)
            s["starts"] = (lens // 4).to(torch.int32).to(DEV)
        else:
            s["starts"] = None
        ends = torch.cat((torch.zeros(1, dtype=torch.int64), count.cumsum(0)))
        s["out_indptr"] = ends.to(torch.int32).to(DEV)
        shape = (int(ends[-1]), c["Hkv"], c["d"])
        dt = torch.float32 if c["f32"] else torch.bfloat16
        s["k_out"], s["v_out"] = (torch.empty(shape, dtype=dt, device=DEV) for _ in range(2))
    else:
        shape = (B, c.get("T", c.get("Tq")), c["Hq"], c["d"])
        s["q"] = torch.randn(shape, device=DEV, generator=gen).to(torch.bfloat16)
        s["out"] = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        s["scale"] = c["d"] ** -0.5
    if own:
        _prepare_own(c, s)
    return s


def _prepare_own(c, s):
    """The handles a program keeps: the layout and the workspace."""
    import split_kv_decode_distattention_gb300 as dattn
    fmt = {"bf16": dattn.KV_BF16, "fp8": dattn.KV_FP8_E4M3, "int4": dattn.KV_INT4,
           "mixed": dattn.KV_MIXED, "fp8-block": dattn.KV_FP8_BLOCK}[c["fmt"]]
    heads = [dattn.KV_INT4 if x else dattn.KV_FP8_E4M3 for x in _four(c["fmt"], c["Hkv"])] \
        if c["fmt"] == "mixed" else None
    s["layout"] = dattn.KVLayout(s["pages"], c["Hkv"], c["d"], c["P"], s["block_table"], fmt,
                                 s["kv_scale"], heads)
    if c["op"] == "shared":
        s["ws"] = dattn.SharedWorkspace(c["sizes"], c["T"], c["Hq"], c["Hkv"], c["d"])
    if c["op"] == "step":
        s["ws"] = dattn.Workspace(c["B"], c["Hq"] * c["T"], c["Hkv"], c["d"])


# ------------------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    return {"shared": _plain_shared, "window": _plain_window, "step": _plain_step,
            "read": _plain_read}[c["op"]](c, state)


def _run_own(c, s):
    import split_kv_decode_distattention_gb300 as dattn
    lay, k, v = s["layout"], s["k_pool"], s["v_pool"]
    if c["op"] == "read":
        dattn.dattn_kv_read(lay, k, v, s["k_out"], s["v_out"], s["out_indptr"], s["seq_lens"],
                            starts=s["starts"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "shared":
        dattn.dattn_decode_shared(lay, k, v, s["q"], s["scale"], s["seq_lens"], s["group_indptr"],
                                  s["prefix_lens"], s["out"], s["ws"])
    elif c["op"] == "window":
        dattn.dattn_prefill_window(lay, k, v, s["q"], s["scale"], s["seq_lens"], c["W"], c["S"],
                                   s["out"])
    else:
        dattn.dattn_decode_window(lay, k, v, s["q"], s["scale"], s["seq_lens"], c["W"], c["S"],
                                  s["out"], s["ws"])
    return s["out"]


def _rows(c, s, at, page, slot):
    """The rows of K (at = 0) or V (1) at (page, slot), fp32: [...][Hkv][d]."""
    Hkv, P, d, fmt = c["Hkv"], c["P"], c["d"], c["fmt"]
    pool = s["v_pool" if at else "k_pool"]
    if fmt == "bf16":
        return pool[page, :, slot].float()
    n = s["pages"]
    if fmt == "fp8-block":
        sc = s["kv_scale"][:n * Hkv * (P // 16) * 2].view(n, Hkv, P // 16, 2)
        x = pool.view(n, Hkv, P, d)[page, :, slot].view(torch.float8_e4m3fn).float()
        return x * sc[page, :, slot // 16, at][..., None]
    sc = s["kv_scale"].view(n, Hkv, P // 16, 2, 16)[page, :, slot // 16, at, slot % 16]
    four = _four(fmt, Hkv)
    h4 = [h for h in range(Hkv) if four[h]]
    h8 = [h for h in range(Hkv) if not four[h]]
    split = n * len(h8) * P * d
    parts = []
    if h8:
        parts.append(pool[:split].view(n, len(h8), P, d)[page, :, slot]
                     .view(torch.float8_e4m3fn).float())
    if h4:
        x = pool[split:].view(n, len(h4), P, d // 2)[page, :, slot]
        parts.append((torch.stack((x & 15, x >> 4), -1).flatten(-2).float() - 8.0))
    x = torch.cat(parts, -2)
    back = torch.tensor(h8 + h4, device=pool.device).argsort()
    return x[..., back, :] * sc[..., None]


def _keys(c, s, at, req, tok):
    """Rows of tokens tok [...] of requests req [...] (broadcast): [...][Hkv][d], fp32."""
    page = s["block_table"].long()[req, (tok // c["P"]).clamp_max(s["block_table"].shape[1] - 1)]
    return _rows(c, s, at, page.clamp_min(0), tok % c["P"])


def _softmax(scores, v):
    """softmax(scores) v over the last axis of scores; rows that see nothing give 0."""
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    e = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(e > 0, e, 1.0)


def _plain_shared(c, s):
    B, T, Hq, d = s["q"].shape
    Hkv, R = c["Hkv"], T * (Hq // c["Hkv"])
    ends, P = s["group_indptr"].long(), s["prefix_lens"].long()
    L = s["seq_lens"].long()
    of = torch.searchsorted(ends, torch.arange(B, device=DEV), right=True) - 1
    q = s["q"].float().view(B, T, Hkv, -1, d).permute(2, 0, 3, 1, 4).reshape(Hkv, B, R, d)
    # every group's prefix once, against the rows of all its requests (padded to the largest group)
    cols = torch.arange(c["sizes"] - c["groups"] + 1, device=DEV)
    member = ends[:-1, None] + cols
    held = member < ends[1:, None]
    member = member.clamp_max(B - 1)
    tok = torch.arange(c["prefix"] // c["P"] * c["P"], device=DEV)
    first = ends[:-1, None]
    k, v = (_keys(c, s, at, first, tok).permute(0, 2, 1, 3) for at in (0, 1))  # [G][Hkv][n][d]
    x = q[:, member].permute(1, 0, 2, 3, 4).reshape(c["groups"], Hkv, -1, d)
    x = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"])
    x.masked_fill_((tok >= P[:, None])[:, None, None], -math.inf)
    m1 = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m1 > -math.inf, m1, 0.0)).exp_()
    e1 = x.sum(-1, keepdim=True)
    o1 = torch.cat((m1, e1, torch.matmul(x, v)), -1)
    o1 = o1.view(c["groups"], Hkv, cols.numel(), R, d + 2).transpose(1, 2)[held]  # [B][Hkv][R]
    m1, e1, o1 = o1[..., :1], o1[..., 1:2], o1[..., 2:]
    # and every request's own tokens
    tok = P[of][:, None] + torch.arange(c["hi"] + c["P"], device=DEV)
    t = torch.arange(T, device=DEV).repeat(Hq // Hkv)  # a row's token
    req = torch.arange(B, device=DEV)[:, None]
    k, v = (_keys(c, s, at, req, tok).permute(0, 2, 1, 3) for at in (0, 1))
    y = torch.matmul(q.transpose(0, 1), k.transpose(2, 3)).mul_(s["scale"])
    seen = tok[:, None, :] <= (L[:, None] - T + t)[..., None]
    y = y.masked_fill_(~seen[:, None], -math.inf)
    m2 = y.amax(-1, keepdim=True)
    m = torch.maximum(m1, m2)
    m = torch.where(m > -math.inf, m, 0.0)
    y = y.sub_(m).exp_()
    f = (m1 - m).exp()
    e = e1 * f + y.sum(-1, keepdim=True)
    o = (o1 * f + torch.matmul(y, v)) / torch.where(e > 0, e, 1.0)
    o = o.view(B, Hkv, Hq // Hkv, T, d).permute(0, 3, 1, 2, 4)
    return o.reshape(B, T, Hq, d).to(torch.bfloat16)


def _plain_window(c, s):
    """Query blocks of C tokens against the window before them, and the first tokens."""
    B, Tq, Hq, d = s["q"].shape
    Hkv, g, W, S = c["Hkv"], Hq // c["Hkv"], c["W"], c["S"]
    C = min(Tq, max(64, min(1024, W)))
    nb = -(-Tq // C)
    L = s["seq_lens"].long()
    t = torch.arange(nb * C, device=DEV).view(nb, C)
    pos = (L - Tq)[:, None, None] + t  # [B][nb][C]
    tok = torch.cat((torch.arange(S, device=DEV).expand(B, nb, S),
                     pos[..., :1] - W + 1 + torch.arange(C + W - 1, device=DEV)), -1)
    near = torch.arange(tok.shape[-1], device=DEV) >= S
    req = torch.arange(B, device=DEV)[:, None, None]
    k, v = (_keys(c, s, at, req, tok.clamp_min(0)).transpose(2, 3) for at in (0, 1))
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, 0, 0, nb * C - Tq)).float()
    q = q.view(B, nb, C, Hkv, g, d).permute(0, 1, 3, 4, 2, 5).reshape(B, nb, Hkv, g * C, d)
    x = torch.matmul(q, k.transpose(3, 4)).mul_(s["scale"]).view(B, nb, Hkv, g, C, -1)
    key, p = tok[:, :, None], pos[..., None]
    seen = (key >= 0) & (key <= p) & torch.where(near, (key > p - W) & (key >= S), key < S)
    x = x.masked_fill_(~seen[:, :, None, None], -math.inf).view(B, nb, Hkv, g * C, -1)
    o = _softmax(x, v).view(B, nb, Hkv, g, C, d).permute(0, 1, 4, 2, 3, 5)
    return o.reshape(B, nb * C, Hq, d)[:, :Tq].to(torch.bfloat16)


def _plain_step(c, s):
    B, T, Hq, d = s["q"].shape
    Hkv, g, W, S = c["Hkv"], Hq // c["Hkv"], c["W"], c["S"]
    W = min(W, c["hi"])
    L = s["seq_lens"].long()
    tok = torch.cat((torch.arange(S, device=DEV).expand(B, S),
                     (L - T - W + 1)[:, None] + torch.arange(W + T - 1, device=DEV)), -1)
    near = torch.arange(tok.shape[-1], device=DEV) >= S
    req = torch.arange(B, device=DEV)[:, None]
    k, v = (_keys(c, s, at, req, tok.clamp_min(0)).transpose(1, 2) for at in (0, 1))
    q = s["q"].float().view(B, T, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * T, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, g, T, -1)
    key, p = tok[:, None], ((L - T)[:, None] + torch.arange(T, device=DEV))[..., None]
    seen = (key >= 0) & (key <= p) & torch.where(near, (key > p - W) & (key >= S), key < S)
    x = x.masked_fill_(~seen[:, None, None], -math.inf).view(B, Hkv, g * T, -1)
    o = _softmax(x, v).view(B, Hkv, g, T, d).permute(0, 3, 1, 2, 4)
    return o.reshape(B, T, Hq, d).to(torch.bfloat16)


def _plain_read(c, s):
    ends = s["out_indptr"].long()
    i = torch.arange(s["k_out"].shape[0], device=DEV)
    req = torch.searchsorted(ends, i, right=True) - 1
    tok = i - ends[req]
    if s["starts"] is not None:
        tok = tok + s["starts"].long()[req]
    dt = s["k_out"].dtype
    return {"k": _keys(c, s, 0, req, tok).to(dt), "v": _keys(c, s, 1, req, tok).to(dt)}


# ------------------------------------------------------------------------------- accounting

def _all_lens(c):
    """Lengths of all requests (a shared prefix among them counted in every one of its requests)."""
    n = c.get("B", c.get("sizes"))
    lens = _spread(c["lo"], c["hi"], n)
    if c["op"] == "shared":
        ends, prefix = _sizes(c)
        of = torch.repeat_interleave(torch.arange(c["groups"]), ends[1:] - ends[:-1])
        lens = lens + prefix[of]
    return lens


def _row_bytes(c):
    """Bytes of a token's K and V rows of all KV heads."""
    if c["fmt"] == "bf16":
        return c["Hkv"] * c["d"] * 4
    codes = 2 * sum(c["d"] // 2 if x else c["d"] for x in _four(c["fmt"], c["Hkv"]))
    return codes + c["Hkv"] * (0.5 if c["fmt"] == "fp8-block" else 8)


def work(case):
    c = case
    L = _all_lens(c).double()
    if c["op"] == "read":
        n = int((_all_lens(c) // 2).clamp_min(1).sum()) if c["middle"] else int(L.sum())
        return {"bytes": n * (_row_bytes(c) + c["Hkv"] * c["d"] * 2 * (4 if c["f32"] else 2)),
                "flops": 2 * n * c["Hkv"] * c["d"]}
    T = c.get("T", c.get("Tq"))
    qo = len(L) * T * c["Hq"] * c["d"] * 4
    if c["op"] == "shared":
        ends, prefix = _sizes(c)
        prefix = (prefix // c["P"] * c["P"]).double()
        n = (ends[1:] - ends[:-1]).double()
        rows = float((L.sum() - (n * prefix).sum()) + prefix.sum())
        seen = float((T * (L - T) + T * (T + 1) / 2).sum())
        return {"bytes": rows * _row_bytes(c) + qo, "flops": 4 * c["Hq"] * c["d"] * seen}
    W, S = c["W"], c["S"]
    p = (L - T)[:, None] + torch.arange(T, dtype=torch.float64)  # positions
    seen = float((torch.minimum(p + 1, torch.tensor(float(W)))
                  + (p + 1 - W).clamp(0, S)).sum())
    rows = float(torch.minimum(L, torch.tensor(float(W + S + T - 1))).sum())
    return {"bytes": rows * _row_bytes(c) + qo, "flops": 4 * c["Hq"] * c["d"] * seen}


# ------------------------------------------------------------------------------- in 64 bits

def _dense64(c, s, b, lo, hi, at):
    """Tokens [lo, hi) of request b in 64 bits, page by page: [Hkv][hi - lo][d]."""
    P, Hkv, d = c["P"], c["Hkv"], c["d"]
    pages = s["block_table"][b, lo // P:-(-hi // P)].long()
    pool, sc = s["v_pool" if at else "k_pool"], s["kv_scale"]
    four = _four(c["fmt"], Hkv)
    n8, n4 = four.count(False), four.count(True)
    out = []
    for h in range(Hkv):
        if c["fmt"] == "bf16":
            x = pool[pages, h].double()
        else:
            n = pool.numel() // (P * (n8 * d + n4 * d // 2))
            mine = four[:h].count(four[h])
            if four[h]:
                y = pool[n * n8 * P * d:].reshape(n, n4, P, d // 2)[pages, mine].int()
                x = torch.empty(len(pages), P, d, dtype=torch.float64, device=pool.device)
                x[..., 0::2], x[..., 1::2] = (y % 16 - 8).double(), (y // 16 - 8).double()
            else:
                y = pool[:n * n8 * P * d].reshape(n, n8, P, d)[pages, mine]
                x = y.view(torch.float8_e4m3fn).double()
            if c["fmt"] == "fp8-block":
                f = sc.double()[:2 * n * Hkv * (P // 16)].reshape(n, Hkv, P // 16, 2)
                f = f[pages, h, :, at].repeat_interleave(16, 1)
            else:
                f = sc.double().reshape(n, Hkv, P // 16, 2, 16)[pages, h, :, at].flatten(1)
            x = x * f[..., None]
        out.append(x.flatten(0, 1)[lo - lo // P * P:][:hi - lo])
    return torch.stack(out)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "read":
        k, v = [], []
        ends = s["out_indptr"].tolist()
        for b in range(c["B"]):
            lo = 0 if s["starts"] is None else int(s["starts"][b])
            for to, at in ((k, 0), (v, 1)):
                to.append(_dense64(c, s, b, lo, lo + ends[b + 1] - ends[b], at).transpose(0, 1))
        return {"k": torch.cat(k), "v": torch.cat(v)}
    T, Hkv, g = s["q"].shape[1], c["Hkv"], c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(s["q"].shape[0]):
        L = int(s["seq_lens"][b])
        for t0 in range(0, T, 1024):
            t1 = min(T, t0 + 1024)
            pos = torch.arange(L - T + t0, L - T + t1, device=DEV)[:, None]
            lo = max(0, L - T + t0 - c["W"] + 1) if "W" in c else 0
            k, v = (_dense64(c, s, b, lo, L - T + t1, at) for at in (0, 1))
            key = torch.arange(lo, L - T + t1, device=DEV)
            see = key[None] <= pos
            if "W" in c:
                first = min(c["S"], lo)  # the first tokens, where the stretch leaves them out
                if first:
                    k, v = (torch.cat((_dense64(c, s, b, 0, first, at), x), 1)
                            for at, x in ((0, k), (1, v)))
                    key = torch.cat((torch.arange(first, device=DEV), key))
                see = (key[None] <= pos) & ((pos - key[None] < c["W"]) | (key[None] < c["S"]))
            for h in range(c["Hq"]):
                w = s["q"][b, t0:t1, h].double() @ k[h // g].T / math.sqrt(c["d"])
                w = torch.softmax(torch.where(see, w, -math.inf), -1)
                out[b, t0:t1, h] = torch.nan_to_num(w, nan=0.0) @ v[h // g]
    return out
