"""The block-scaled 8-bit pool on the GPU: what the append stores, bit for bit, and the attention
over it against a 64-bit softmax over the reference's own values.

The attention's tolerance is the bound that _block_ref.attention derives, row by row; m and e
follow from the same logit error (m: the error itself; e: its relative size).
"""
import numpy as np
import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import workloads as W
from split_kv_decode_distattention_gb300.harness import PagedCache

import _block_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BLOCK = dattn.KV_FP8_BLOCK


def _cache(case, fill=False, stats=False, junk=False, **kw):
    c = PagedCache(case, DEV, with_stats=stats, kv_format=BLOCK, fill=fill, zero_pool=True, **kw)
    if junk:  # what recycled pages may hold: NaN codes and any scale
        c.k_pool.fill_(0x7F)
        c.v_pool.fill_(0xFF)
        c.kv_scale.fill_(float("nan"))
    return c


def _pools(case, junk=False):
    a = dict(codes=0x7F, scale=float("nan")) if junk else {}
    b = dict(codes=0xFF, scale=float("nan")) if junk else {}
    n = (case.num_pages, case.Hkv, case.P, case.d)
    return ref.BlockPool(*n, **a), ref.BlockPool(*n, **b)


def _assert_pool(cache, kp, vp):
    torch.cuda.synchronize()
    np.testing.assert_array_equal(cache.k_pool.cpu().numpy(), kp.codes)
    np.testing.assert_array_equal(cache.v_pool.cpu().numpy(), vp.codes)
    n = kp.scale.size
    sc = cache.kv_scale[:2 * n].cpu().numpy().reshape(*kp.scale.shape, 2)
    np.testing.assert_array_equal(sc[..., 0].view(np.uint32), kp.scale.view(np.uint32))
    np.testing.assert_array_equal(sc[..., 1].view(np.uint32), vp.scale.view(np.uint32))


def _rows(shape, seed, spread=0):
    """bf16 rows; spread > 0: each token has its own power-of-two size."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape).astype(np.float32)
    if spread:
        x *= np.exp2(rng.integers(-spread, spread + 1, size=(*shape[:2], 1, 1))).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("d,P", [(128, 16), (64, 64), (128, 80), (64, 256)])
def test_append_stores_the_formats_codes_and_scales(d, P):
    """Single tokens, windows and long chunks, tokens of very different sizes: scales are raised
    and earlier codes rounded again; recycled pages' contents take no part."""
    case = W.Case("blk", B=3, Hq=3, Hkv=3, d=d, P=P, lens=[0, 0, 0], seed=3, reserve_tokens=420)
    cache = _cache(case, junk=True)
    kp, vp = _pools(case, junk=True)
    for step, T in enumerate([1, 1, 13, 1, 40, 1, 7, 230, 1, 1]):
        k, v = _rows((3, T, 3, d), 10 + step, 9), _rows((3, T, 3, d), 90 + step, 3)
        for b in range(3):
            for pool, x in ((kp, k), (vp, v)):
                pool.append(case.block_table[b], cache.lens[b], x[b].double().cpu().numpy())
        cache.append(k, v)
        _assert_pool(cache, kp, vp)
    assert int(cache.dev_err.item()) == 0


def test_append_of_corner_values():
    """Zeros of both signs, a scale's border (448 and the next bf16 value), E4M3 ties and
    subnormals, the smallest and largest bf16 values, infinities and NaN."""
    d = 64
    x = torch.zeros(20, 1, d)
    x[1, 0, :] = -0.0
    x[2, 0, 0], x[3, 0, 0] = 448.0, 450.0
    x[4, 0, :] = 1.0625
    x[5, 0, :8] = torch.tensor([2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -10, 2.0 ** -11, -2.0 ** -10,
                                3 * 2.0 ** -10, 5 * 2.0 ** -10, 7 * 2.0 ** -10])
    x[6, 0, 0] = 2.0 ** -133  # a subnormal bf16 value
    x[7, 0, 0] = 3.3895313892515355e38
    x = x.to(torch.bfloat16).to(DEV)
    for order in ([0, 1], [2], [3], [2, 3], [4], [5, 2], [6], [6, 0, 4], [7], [5, 4, 3, 7],
                  [0, 6, 5, 4, 2, 3, 7]):
        case = W.Case("corner", B=1, Hq=1, Hkv=1, d=d, P=16, lens=[0], seed=1)
        cache, (kp, vp) = _cache(case, junk=True), _pools(case, junk=True)
        for i in order:  # one by one
            row = x[i].view(1, 1, 1, d)
            cache.append(row, -row)
            kp.append(case.block_table[0], cache.lens[0] - 1, x[i].double().cpu().numpy()[None])
            vp.append(case.block_table[0], cache.lens[0] - 1, -x[i].double().cpu().numpy()[None])
            _assert_pool(cache, kp, vp)
        one, (kp, vp) = _cache(case, junk=True), _pools(case, junk=True)  # in one call
        rows = x[order].view(1, len(order), 1, d)
        one.append(rows, -rows)
        kp.append(case.block_table[0], 0, x[order].double().cpu().numpy())
        vp.append(case.block_table[0], 0, -x[order].double().cpu().numpy())
        _assert_pool(one, kp, vp)
    # infinities saturate, a NaN stays one and does not enter the scale
    case = W.Case("inf", B=1, Hq=1, Hkv=1, d=d, P=16, lens=[0], seed=1)
    cache = _cache(case)
    k = torch.ones(1, 2, 1, d, dtype=torch.bfloat16, device=DEV)
    k[0, 0, 0, 0], k[0, 1, 0, 1] = float("inf"), float("nan")
    cache.append(k, k)
    torch.cuda.synchronize()
    page = int(case.block_table[0, 0])
    codes = cache.k_pool[page, 0].cpu().numpy()
    assert codes[0, 0] == 0x7E and codes[1, 1] & 0x7F == 0x7F and codes[0, 1] == 0
    assert cache.kv_scale.view(-1, 2)[page, 0].item() == 2.0 ** 119


def test_append_statistics_are_the_keys():
    """k_max and k_min come from the bf16 keys, as for the other pools."""
    case = W.Case("st", B=2, Hq=2, Hkv=2, d=64, P=32, lens=[50, 19], seed=5)
    a = _cache(case, fill=True, stats=True)
    b = PagedCache(case, DEV, with_stats=True, zero_pool=True)
    for T in (1, 30, 1):
        k, v = a.new_tokens(T)
        a.append(k, v)
        b.append(k, v)
    torch.cuda.synchronize()
    assert torch.equal(a.stats.view(torch.int16), b.stats.view(torch.int16))


# ---------------------------------------------------------------- attention

def _filled(case, seed, stats=False, junk=True, steps=(1.0,)):
    """A cache filled request by request, and the reference's pools."""
    cache, (kp, vp) = _cache(case, stats=stats, junk=junk), _pools(case, junk)
    for b, L in enumerate(case.lens):
        if L == 0:
            continue
        k = _rows((1, L, case.Hkv, case.d), seed + b, 2)
        v = _rows((1, L, case.Hkv, case.d), seed + 50 + b, 2)
        at = 0
        for part in (L - L // 3, L // 3):  # two calls: a block is extended
            if part == 0:
                continue
            ks, vs = k[:, at:at + part].contiguous(), v[:, at:at + part].contiguous()
            dattn.dattn_kv_append(cache._row_layout(b), cache.k_pool, cache.v_pool, cache.stats,
                                  ks, vs, cache.seq_lens[b:b + 1], cache.dev_err)
            kp.append(case.block_table[b], at, ks[0].double().cpu().numpy())
            vp.append(case.block_table[b], at, vs[0].double().cpu().numpy())
            at += part
        cache.lens[b] = L
    _assert_pool(cache, kp, vp)
    return cache, kp, vp


def _check(case, q, out, m, e, kp, vp, see_of=None, weights=2.0 ** -20):
    """q, out [B][T][Hq][d]; see_of(b, kvh) -> [T][L] visible keys (default: causal)."""
    B, T, Hq, d = q.shape
    q64, o = q.double().cpu().numpy(), out.double().cpu().numpy()
    mm, ee = (None if t is None else t.double().cpu().numpy() for t in (m, e))
    for b in range(B):
        L = case.lens[b]
        K, V = kp.values(case.block_table[b], L), vp.values(case.block_table[b], L)
        causal = np.arange(L)[None] <= (L - T + np.arange(T))[:, None]
        for h in range(Hq):
            kvh = h // case.g
            see = causal if see_of is None else see_of(b, kvh)
            w, wm, we, tol, t = ref.attention(q64[b, :, h], K[:, kvh], V[:, kvh], case.scale, see,
                                                weights)
            err = np.abs(o[b, :, h] - w).max(-1)
            assert (err <= tol + 2.0 ** -23 * np.abs(w).max(-1, initial=0.0)).all(), (
                b, h, L, err, tol)
            if mm is not None:
                none = ~np.isfinite(wm)
                assert (mm[b, none, h] == -np.inf).all() and (ee[b, none, h] == 0).all()
                ok = ~none
                assert (np.abs(mm[b, ok, h] - wm[ok]) <= t[ok] + 2.0 ** -22 * np.abs(wm[ok])).all()
                assert (np.abs(ee[b, ok, h] / we[ok] - 1) <= 2 * t[ok] + 2.0 ** -20).all()


CASES = [
    # B, Hq, Hkv, d, P, lens
    (4, 4, 4, 128, 16, [1, 0, 17, 300]),
    (3, 16, 2, 128, 64, [64, 63, 1000]),
    (2, 6, 2, 64, 48, [2000, 5]),
    (2, 8, 4, 64, 256, [257, 511]),
    (1, 5, 1, 128, 16, [3333]),
]


@pytest.mark.parametrize("B,Hq,Hkv,d,P,lens", CASES)
@pytest.mark.parametrize("splits", [0, 1, 13])
def test_decode_over_the_block_scaled_pool(B, Hq, Hkv, d, P, lens, splits):
    case = W.Case("dec", B=B, Hq=Hq, Hkv=Hkv, d=d, P=P, lens=lens, seed=6)
    cache, kp, vp = _filled(case, 7)
    q = _rows((B, 1, Hq, d), 77)
    out = torch.full((B, Hq, d), float("nan"), device=DEV)
    m, e = torch.full((B, Hq), float("nan"), device=DEV), torch.full((B, Hq), float("nan"),
                                                                    device=DEV)
    ws = cache.workspace(num_splits=splits)
    for _ in range(2):
        cache.decode(q[:, 0].contiguous(), out, ws, m, e, num_splits=splits)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    _check(case, q, out[:, None], m[:, None], e[:, None], kp, vp)


@pytest.mark.parametrize("T,Hq,Hkv", [(2, 8, 2), (3, 2, 2), (8, 2, 2)])
def test_multi_query_decode_over_the_block_scaled_pool(T, Hq, Hkv):
    case = W.Case("multi", B=3, Hq=Hq, Hkv=Hkv, d=128, P=32, lens=[T, 200, 16 + T - 1], seed=6)
    cache, kp, vp = _filled(case, 8)
    q = _rows((3, T, Hq, 128), 78)
    out = torch.empty(3, T, Hq, 128, device=DEV)
    m, e = torch.empty(3, T, Hq, device=DEV), torch.empty(3, T, Hq, device=DEV)
    cache.decode(q, out, cache.workspace(queries=T), m, e)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    _check(case, q, out, m, e, kp, vp)


def test_partials_over_the_block_scaled_pool_merge_to_the_whole():
    case = W.Case("part", B=2, Hq=4, Hkv=2, d=128, P=16, lens=[700, 90], seed=6)
    cache, kp, vp = _filled(case, 9)
    q = _rows((2, 1, 4, 128), 79)
    sets = [case.page_sets_of(b, case.lens[b]) for b in range(2)]
    req = torch.tensor([b for b in range(2) for _ in sets[b]], dtype=torch.int32, device=DEV)
    flat = [s for b in range(2) for s in sets[b]]
    ind = torch.tensor(np.cumsum([0] + [len(s) for s in flat]), dtype=torch.int32, device=DEV)
    pages = torch.tensor(np.concatenate(flat), dtype=torch.int32, device=DEV)
    C = len(flat)
    m, e, MA = (torch.empty(*s, device=DEV) for s in ((C, 4), (C, 4), (C, 4, 128)))
    ws = dattn.Workspace(C, 4, 2, 128)
    dattn.dattn_partial(cache.layout, cache.k_pool, cache.v_pool, q[:, 0].contiguous(), case.scale,
                        cache.seq_lens, req, ind, pages, m, e, MA, ws, dev_err=cache.dev_err)
    out = torch.empty(2, 4, 128, device=DEV)
    heads = torch.tensor([0, len(sets[0]), C], dtype=torch.int32, device=DEV)
    dattn.dattn_merge(heads, m, e, MA, out=out, dev_err=cache.dev_err)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    _check(case, q, out[:, None], None, None, kp, vp)


def test_block_sparse_decode_over_the_block_scaled_pool():
    kinds = [W.HEAD_RETRIEVAL, W.HEAD_STREAMING, W.HEAD_DENSE]
    case = W.Case("sparse", B=2, Hq=6, Hkv=3, d=64, P=64, lens=[1500, 70], seed=6, head_kind=kinds,
                  top_k=5, sinks=4, local=24)
    cache, kp, vp = _filled(case, 11, stats=True)
    q = _rows((2, 1, 6, 64), 80)
    sel = torch.empty(2, 3, 5, dtype=torch.int32, device=DEV)
    cache.select(q[:, 0].contiguous(), sel, cache.workspace(top_k=5))
    out = torch.empty(2, 6, 64, device=DEV)
    cache.decode(q[:, 0].contiguous(), out, cache.workspace(), sparse=cache.sparse_config(sel))
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0

    def see_of(b, kvh):
        t = np.arange(case.lens[b])
        if kinds[kvh] == W.HEAD_RETRIEVAL:
            return np.isin(t // 64, sel[b, kvh].cpu().numpy())[None]
        if kinds[kvh] == W.HEAD_STREAMING:
            return ((t < 4) | (t >= max(4, case.lens[b] - 24)))[None]
        return np.ones((1, case.lens[b]), bool)

    _check(case, q, out[:, None], None, None, kp, vp, see_of)


def test_block_scales_of_every_size_in_one_sequence():
    """Tiles whose V scales span 2^-100 .. 2^100 in any order, and tiles of zeros: the running
    scale of the weighted sum is raised, and a tile far below it adds nothing."""
    d, n = 64, 12
    case = W.Case("range", B=1, Hq=2, Hkv=1, d=d, P=16, lens=[16 * n], seed=2)
    cache, (kp, vp) = _cache(case, junk=True), _pools(case, junk=True)
    k, v = _rows((1, 16 * n, 1, d), 1), _rows((1, 16 * n, 1, d), 2)
    ex = [0, -100, 30, 3, -40, 100, 99, 0, -126, 60, 100, -3]
    for i, x in enumerate(ex):
        v[:, 16 * i:16 * i + 16] *= 2.0 ** x
    v[:, 112:128] = 0
    k[:, 32:48] = 0
    cache.append(k, v)
    kp.append(case.block_table[0], 0, k[0].double().cpu().numpy())
    vp.append(case.block_table[0], 0, v[0].double().cpu().numpy())
    _assert_pool(cache, kp, vp)
    q = _rows((1, 1, 2, d), 3)
    for splits in (1, 3):
        out = torch.empty(1, 2, d, device=DEV)
        cache.decode(q[:, 0].contiguous(), out, cache.workspace(num_splits=splits),
                     num_splits=splits)
        torch.cuda.synchronize()
        _check(case, q, out[:, None], None, None, kp, vp)


def test_a_step_appends_with_rotation_and_decodes():
    """The operators together as a decode loop uses them, captured once and replayed: rotate and
    append, then decode over the block-scaled pool."""
    r = dattn.Rotation(128, base=500000.0)
    case = W.Case("step", B=3, Hq=8, Hkv=2, d=128, P=16, lens=[5, 100, 31], seed=6)
    cache, kp, vp = _filled(case, 13)
    q, k, v = (torch.empty(3, 1, h, 128, dtype=torch.bfloat16, device=DEV) for h in (8, 2, 2))
    qr, out, ws = torch.empty_like(q), torch.empty(3, 8, 128, device=DEV), cache.workspace()
    lens = list(case.lens)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        dattn.dattn_rope_append(cache.layout, cache.k_pool, cache.v_pool, None, r, q, k, v, qr,
                                cache.seq_lens, dev_err=cache.dev_err)
        cache.decode(qr[:, 0], out, ws)
    for step in range(4):
        for i, t in enumerate((q, k, v)):
            t.copy_(_rows(t.shape, 200 + 3 * step + i))
        pos = cache.seq_lens.clone()
        g.replay()
        kr, want_q = torch.empty_like(k), torch.empty_like(q)
        dattn.dattn_rope(r, k, kr, pos)
        dattn.dattn_rope(r, q, want_q, pos)
        torch.cuda.synchronize()
        assert torch.equal(qr, want_q)
        for b in range(3):
            kp.append(case.block_table[b], lens[b], kr[b].double().cpu().numpy())
            vp.append(case.block_table[b], lens[b], v[b].double().cpu().numpy())
        lens = [n + 1 for n in lens]
        case.lens = lens
        assert cache.seq_lens.tolist() == lens and int(cache.dev_err.item()) == 0
        _assert_pool(cache, kp, vp)
        _check(case, qr, out[:, None], None, None, kp, vp)


# ---------------------------------------------------------------- prefill

# the weights enter the products as two bf16 terms: half a step of half a step, 2^-18, beside 2^-20
PREFILL = 2.0 ** -18 + 2.0 ** -20


def _prefill(cache, q, sparse=None, out=None):
    B, Tq, Hq, d = q.shape
    out = torch.full((B, Tq, Hq, d), float("nan"), device=DEV) if out is None else out
    m, e = (torch.full((B, Tq, Hq), float("nan"), device=DEV) for _ in range(2))
    dattn.dattn_prefill(cache.layout, cache.k_pool, cache.v_pool, q, cache.case.scale,
                        cache.seq_lens, out, m, e, sparse=sparse, dev_err=cache.dev_err)
    torch.cuda.synchronize()
    return out, m, e


PREFILL_CASES = [
    # Hq, Hkv, d, P, lens, Tq
    (4, 1, 128, 16, [64], 64),          # one query block of four heads
    (4, 1, 64, 16, [1, 77, 300], 1),    # single tokens
    (8, 2, 128, 64, [129, 70, 500], 70),
    (2, 2, 128, 16, [300, 700], 280),   # one head: four query blocks, some past the chunk
    (6, 3, 64, 48, [200, 131], 131),    # pairs of heads
    (3, 1, 64, 256, [513], 200),
    (8, 1, 128, 32, [100, 999], 33),
    (5, 5, 64, 16, [64, 65], 2),
]


@pytest.mark.parametrize("Hq,Hkv,d,P,lens,Tq", PREFILL_CASES)
def test_causal_prefill_over_the_block_scaled_pool(Hq, Hkv, d, P, lens, Tq):
    case = W.Case("pf", B=len(lens), Hq=Hq, Hkv=Hkv, d=d, P=P, lens=lens, seed=6)
    cache, kp, vp = _filled(case, 21)
    q = _rows((len(lens), Tq, Hq, d), 81)
    out, m, e = _prefill(cache, q)
    assert int(cache.dev_err.item()) == 0
    _check(case, q, out, m, e, kp, vp, weights=PREFILL)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 64), (12, 3, 128), (6, 3, 128), (3, 3, 128)])
def test_block_sparse_prefill_over_the_block_scaled_pool(Hq, Hkv, d):
    kinds = [W.HEAD_RETRIEVAL, W.HEAD_STREAMING, W.HEAD_DENSE, W.HEAD_RETRIEVAL][:Hkv]
    lens, Tq = [900, 450], 333
    case = W.Case("pfs", B=2, Hq=Hq, Hkv=Hkv, d=d, P=32, lens=lens, seed=6)
    cache, kp, vp = _filled(case, 22)
    stride, max_sel = 15, 9
    rng = np.random.default_rng(3)
    lists = np.full((2, Hkv, stride, max_sel), -1, np.int32)
    for row in lists.reshape(-1, max_sel):
        n = rng.integers(0, max_sel + 1)
        row[:n] = rng.permutation(17)[:n]  # blocks after the query's too
    lists[0, 0, 11] = -1  # queries that keep nothing
    sp = dattn.PrefillSparseConfig(torch.tensor(kinds, dtype=torch.int8, device=DEV), 1, 2,
                                   torch.from_numpy(lists).to(DEV))
    q = _rows((2, Tq, Hq, d), 82)
    out, m, e = _prefill(cache, q, sp)
    assert int(cache.dev_err.item()) == 0

    def see_of(b, kvh):
        L = lens[b]
        key, pos = np.arange(L)[None], (L - Tq + np.arange(Tq))[:, None]
        kb, qb = key // 64, pos // 64
        keep = key <= pos
        if kinds[kvh] == W.HEAD_STREAMING:
            return keep & ((kb < 1) | (kb > qb - 2))
        if kinds[kvh] == W.HEAD_RETRIEVAL:
            held = (lists[b, kvh][:, :, None] == np.arange(17)).any(1)
            return keep & held[qb, kb]
        return keep

    _check(case, q, out, m, e, kp, vp, see_of, weights=PREFILL)


def test_prefill_with_scales_of_every_size():
    """Blocks whose scales span 2^-100 .. 2^100 (above and below what one bf16 factor reaches)."""
    d, n = 128, 16
    case = W.Case("pfr", B=1, Hq=4, Hkv=1, d=d, P=16, lens=[16 * n], seed=2)
    cache, (kp, vp) = _cache(case, junk=True), _pools(case, junk=True)
    k, v = _rows((1, 16 * n, 1, d), 1), _rows((1, 16 * n, 1, d), 2)
    for i, x in enumerate([0, -100, 30, 3, -40, 100, 99, 0, -126, 60, 100, -3, 15, 16, 17, 8]):
        v[:, 16 * i:16 * i + 16] *= 2.0 ** x
        k[:, 16 * i:16 * i + 16] *= 2.0 ** (-x if x > 40 else min(x, 0))
    k[:, 32:48] = 0
    cache.append(k, v)
    kp.append(case.block_table[0], 0, k[0].double().cpu().numpy())
    vp.append(case.block_table[0], 0, v[0].double().cpu().numpy())
    q = _rows((1, 70, 4, d), 3)
    out, m, e = _prefill(cache, q)
    assert int(cache.dev_err.item()) == 0
    _check(case, q, out, m, e, kp, vp, weights=PREFILL)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_prefill_with_other_softmax_scales(scale):
    case = W.Case("pfn", B=1, Hq=2, Hkv=1, d=64, P=16, lens=[190], seed=6, scale=scale or 1.0)
    case.scale = scale
    cache, kp, vp = _filled(case, 23)
    q = _rows((1, 100, 2, 64), 83)
    out, m, e = _prefill(cache, q)
    _check(case, q, out, m, e, kp, vp, weights=PREFILL)


def test_prefill_flags_bad_pages_and_lengths():
    """An unmapped page adds nothing, a length below Tq leaves its request's outputs alone."""
    case = W.Case("pfb", B=3, Hq=4, Hkv=1, d=64, P=16, lens=[200, 200, 90], seed=6)
    cache, kp, vp = _filled(case, 24)
    q = _rows((3, 100, 4, 64), 84)
    want, _, _ = _prefill(cache, q[:2].contiguous())
    lay = cache.layout
    cache.block_table[0, 2] = -1
    cache.block_table[0, 5] = case.num_pages + 3
    out = torch.full((3, 100, 4, 64), 9.0, device=DEV)
    _prefill(cache, q, out=out)
    E = dattn.DEVERR
    assert int(cache.dev_err.item()) == E["UNMAPPED_PAGE"] | E["PAGE_OOB"] | E["LEN_OOB"]
    assert (out[2] == 9.0).all()
    assert torch.equal(out[1], want[1])
    hole = np.isin(np.arange(200) // 16, [2, 5])
    case.lens = case.lens[:1]

    def see_of(b, kvh):
        return (np.arange(200)[None] <= (100 + np.arange(100))[:, None]) & ~hole[None]

    _check(case, q[:1], out[:1], None, None, kp, vp, see_of, weights=PREFILL)


def test_prefill_agrees_with_decode_and_repeats():
    """Tq = 1 over a long context is a decode; the same call gives the same bits again, after
    another context's call and in a captured graph."""
    case = W.Case("pfd", B=2, Hq=16, Hkv=4, d=128, P=16, lens=[5000, 2222], seed=6)
    cache, kp, vp = _filled(case, 25)
    q = _rows((2, 1, 16, 128), 85)
    out, m, e = _prefill(cache, q)
    _check(case, q, out, m, e, kp, vp, weights=PREFILL)
    dec = torch.empty(2, 16, 128, device=DEV)
    cache.decode(q[:, 0].contiguous(), dec, cache.workspace())
    torch.cuda.synchronize()
    _check(case, q, dec[:, None], None, None, kp, vp)
    g = torch.cuda.CUDAGraph()
    again = torch.empty_like(out)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        dattn.dattn_prefill(cache.layout, cache.k_pool, cache.v_pool, q, case.scale,
                            cache.seq_lens, again, dev_err=cache.dev_err)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    assert int(cache.dev_err.item()) == 0


def test_other_quantized_pools_still_have_no_prefill():
    case = W.Case("no", B=1, Hq=2, Hkv=2, d=64, P=16, lens=[20], seed=6)
    for fmt in (dattn.KV_FP8_E4M3, dattn.KV_INT4):
        c = PagedCache(case, DEV, kv_format=fmt, zero_pool=True)
        q = _rows((1, 4, 2, 64), 86)
        with pytest.raises(dattn.DattnError, match="UNSUPPORTED"):
            _prefill(c, q)


def _filled_fast(case, seed):
    """A cache filled through the append, without the reference's pools, and its values in 64 bits
    read from the codes on the GPU: [B][Hkv][L][d] of K and V (request 0)."""
    cache = _cache(case)
    L = case.lens[0]
    k, v = _rows((1, L, case.Hkv, case.d), seed), _rows((1, L, case.Hkv, case.d), seed + 1)
    cache.append(k, v)
    n = case.num_pages * case.Hkv * (case.P // 16)
    sc = cache.kv_scale[:2 * n].view(case.num_pages, case.Hkv, case.P // 16, 2).double()
    pages = cache.block_table[0, :-(-L // case.P)].long()
    out = []
    for i, pool in enumerate((cache.k_pool, cache.v_pool)):
        x = pool.view(torch.float8_e4m3fn)
        x = x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
        x = x * sc[pages][..., i].repeat_interleave(16, 2)[..., None]
        out.append(x.transpose(0, 1).reshape(case.Hkv, -1, case.d)[:, :L])
    return cache, out[0], out[1]


def _attention64(q, K, V, scale):
    """q [T][Hq][d] (the last T tokens) over K, V [Hkv][L][d], causal, on the GPU in 64 bits."""
    T, Hq, d = q.shape
    Hkv, L, _ = K.shape
    out = torch.empty(T, Hq, d, dtype=torch.float64, device=DEV)
    see = torch.arange(L, device=DEV)[None] <= (L - T + torch.arange(T, device=DEV))[:, None]
    for h in range(Hq):
        w = (q[:, h].double() @ K[h * Hkv // Hq].T * scale).masked_fill_(~see, -np.inf)
        out[:, h] = torch.softmax(w, -1) @ V[h * Hkv // Hq]
    return out


@pytest.mark.parametrize("Hq,Hkv,d,Tq,L", [(32, 8, 128, 1400, 9000), (16, 16, 64, 700, 7001),
                                           (12, 6, 128, 1100, 5000)])
def test_long_prefill_of_many_tiles(Hq, Hkv, d, Tq, L):
    """Enough tiles for whole waves and single tiles, enough key blocks for several emptyings of
    the accumulators (every 32). Between two of them a sum takes in 256 products, each losing less
    than 2^-23 of it: 2^-15 together, beside which the other errors vanish. A repeated call gives
    the same bits, and so does one beside another call on another stream."""
    case = W.Case("pfl", B=1, Hq=Hq, Hkv=Hkv, d=d, P=16, lens=[L], seed=6)
    cache, K, V = _filled_fast(case, 31)
    q = _rows((1, Tq, Hq, d), 87)
    out, m, e = _prefill(cache, q)
    want = _attention64(q[0], K, V, case.scale)
    assert ((out[0] - want).norm() / want.norm()).item() <= 2.0 ** -15
    for h in (0, Hq - 1):  # no single row far off
        err = (out[0, :, h] - want[:, h]).norm(dim=1) / want[:, h].norm(dim=1)
        assert err.max().item() <= 2.0 ** -14
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.empty_like(out) for _ in streams]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        for _ in range(2):
            dattn.dattn_prefill(cache.layout, cache.k_pool, cache.v_pool, q, case.scale,
                                cache.seq_lens, o, dev_err=cache.dev_err, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
    assert int(cache.dev_err.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,d,Tq,L", [(32, 8, 128, 64, 9000), (8, 1, 64, 1, 20001),
                                           (16, 16, 128, 33, 5000), (6, 3, 128, 130, 3001),
                                           (12, 4, 64, 100, 4097), (4, 1, 128, 300, 300)])
def test_prefill_of_few_rows_over_a_long_context(Hq, Hkv, d, Tq, L):
    """Few tiles: clusters of CTAs share a tile's key blocks (more than 32 each in the first two, so
    that accumulators are emptied). Errors as above; repeated and captured calls give the same bits."""
    case = W.Case("pff", B=1, Hq=Hq, Hkv=Hkv, d=d, P=16, lens=[L], seed=6)
    cache, K, V = _filled_fast(case, 33)
    q = _rows((1, Tq, Hq, d), 88)
    out, m, e = _prefill(cache, q)
    want = _attention64(q[0], K, V, case.scale)
    err = (out[0] - want).norm(dim=2) / want.norm(dim=2)
    assert err.max().item() <= 2.0 ** -14 and ((out[0] - want).norm() / want.norm()) <= 2.0 ** -15
    # m + ln e is the logarithm of the sum: scores of a few units, 2^-18 of them and of the sum
    see = torch.arange(L, device=DEV)[None] <= (L - Tq + torch.arange(Tq, device=DEV))[:, None]
    for h in (0, Hq - 1):
        w = (q[0, :, h].double() @ K[h * Hkv // Hq].T * case.scale).masked_fill_(~see, -np.inf)
        top, lse = w.max(1).values, torch.logsumexp(w, 1)
        assert ((m[0, :, h] - top).abs() <= 2.0 ** -18 * (1 + top.abs())).all()
        assert ((m[0, :, h] + e[0, :, h].double().log() - lse).abs() <= 2.0 ** -16).all()
    again = torch.empty_like(out)
    call = lambda: dattn.dattn_prefill(cache.layout, cache.k_pool, cache.v_pool, q,  # noqa: E731
                                       case.scale, cache.seq_lens, again, dev_err=cache.dev_err)
    call()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    again.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out) and int(cache.dev_err.item()) == 0


def test_prefill_of_few_rows_beside_empty_and_bad_requests():
    """Short, zero-length and over-long requests beside a long one in clusters of four; rows of
    a request that the call refuses stay as they were."""
    lens = [1500, 9, 40, 700]
    case = W.Case("pfb", B=4, Hq=4, Hkv=1, d=64, P=16, lens=lens, seed=6)
    cache, kp, vp = _filled(case, 24)
    q = _rows((4, 9, 4, 64), 89)
    want, m, e = _prefill(cache, q)
    _check(case, q, want, m, e, kp, vp, weights=PREFILL)
    cache.seq_lens[1], cache.seq_lens[3] = 0, 16 * case.max_pages + 1
    out = torch.full_like(want, 7.0)
    out, _, _ = _prefill(cache, q, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    assert (out[1] == 7.0).all() and (out[3] == 7.0).all()
    assert int(cache.dev_err.item()) != 0


def test_prefill_whose_row_maxima_climb():
    """Keys whose scores climb by 2^9 and more from window to window and block to block: what the
    output row holds of earlier windows is moved to the new reference, or vanishes beside it."""
    d, L, Tq = 64, 64 * 100, 64
    case = W.Case("pfc", B=1, Hq=4, Hkv=1, d=d, P=64, lens=[L], seed=6, scale=1.0)
    cache, kp, vp = _cache(case), *_pools(case)
    k, v = _rows((1, L, 1, d), 41), _rows((1, L, 1, d), 42)
    q = torch.zeros(1, Tq, 4, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = torch.tensor([1.0, 0.02, 3.0, -1.0], device=DEV).to(torch.bfloat16)
    k[0, :, 0, 0] = (torch.arange(L, device=DEV) // 64 * 8).to(torch.bfloat16)
    cache.append(k, v)
    kp.append(case.block_table[0], 0, k[0].double().cpu().numpy())
    vp.append(case.block_table[0], 0, v[0].double().cpu().numpy())
    out, m, e = _prefill(cache, q)
    _check(case, q, out, m, e, kp, vp, weights=PREFILL)


def test_prefill_of_many_tiles_whose_row_maxima_climb():
    """As above with a CTA for each tile pair or tile, and no clusters."""
    d, L, Tq, Hkv = 64, 64 * 70, 128, 20
    case = W.Case("pfm", B=1, Hq=4 * Hkv, Hkv=Hkv, d=d, P=64, lens=[L], seed=6, scale=1.0)
    cache, kp, vp = _cache(case), *_pools(case)
    k, v = _rows((1, L, Hkv, d), 43), _rows((1, L, Hkv, d), 44)
    q = torch.zeros(1, Tq, 4 * Hkv, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = torch.tensor([1.0, 0.02, 3.0, -1.0], device=DEV).to(torch.bfloat16).repeat(Hkv)
    k[0, :, :, 0] = (torch.arange(L, device=DEV) // 64 * 8).to(torch.bfloat16)[:, None]
    cache.append(k, v)
    kp.append(case.block_table[0], 0, k[0].double().cpu().numpy())
    vp.append(case.block_table[0], 0, v[0].double().cpu().numpy())
    out, m, e = _prefill(cache, q)
    _check(case, q, out, m, e, kp, vp, weights=PREFILL)


def test_decode_over_a_long_context_keeps_its_precision():
    """32K keys: a tile's weighted sum is added rounding to nearest, 2^-24 of the sum a tile in any
    order, random in sign: under 2^-20 of the output's norm."""
    case = W.Case("dl", B=1, Hq=8, Hkv=2, d=128, P=16, lens=[32768], seed=6)
    cache, K, V = _filled_fast(case, 33)
    q = _rows((1, 1, 8, 128), 88)
    out = torch.empty(1, 8, 128, device=DEV)
    cache.decode(q[:, 0].contiguous(), out, cache.workspace(num_splits=1), num_splits=1)
    want = _attention64(q[0], K, V, case.scale)
    assert ((out - want).norm() / want.norm()).item() <= 2.0 ** -20
