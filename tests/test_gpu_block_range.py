"""Attention over the block-scaled 8-bit pool where V scales differ by powers of two that the weights'
own formats do not span: what a row does not see, or gives no weight to, takes nothing from it.

The reference is a 64-bit softmax over the values that the pool holds (its codes times its scales),
and each element of a row is bounded by what the row itself sees:
    |error| <= t (sum_i p_i |V_i| + |out|) + 2^-33 max_j(p_j s_j) sum_i |V_i| / s_i
with t the relative error of a weight (its logit: d * 2^-23 of the sum of magnitudes; exponential and
rounding: 2^-20) and of the weighted sum (two products for 16 keys, each less than 2^-23 of the sum of
magnitudes). The second term is what a weight below the smallest steps of its two 16-bit terms may
lose: 2^-25 of a unit in which the row's largest weight times V scale s_j, over the keys that it sees and
whose V is not all zeros, is 2^8 or more.
"""
import numpy as np
import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import workloads as W
from split_kv_decode_distattention_gb300.harness import PagedCache

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _rows(shape, seed):
    x = np.random.default_rng(seed).normal(size=shape).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).to(DEV)


def _cache(case):
    return PagedCache(case, DEV, kv_format=dattn.KV_FP8_BLOCK, fill=False, zero_pool=True)


def _held(cache, b, L):
    """What the pool holds of request b: K and V values [Hkv][L][d] and V scales [Hkv][L], 64 bits."""
    c = cache.case
    n = c.num_pages * c.Hkv * (c.P // 16)
    sc = cache.kv_scale[:2 * n].view(c.num_pages, c.Hkv, c.P // 16, 2).double()
    pages = cache.block_table[b, :-(-L // c.P)].long()
    out = []
    for i, pool in enumerate((cache.k_pool, cache.v_pool)):
        x = pool[pages].view(torch.float8_e4m3fn).double()
        s = sc[pages][..., i].repeat_interleave(16, 2)
        out.append((x * s[..., None]).transpose(0, 1).reshape(c.Hkv, -1, c.d)[:, :L])
        out.append(s.transpose(0, 1).reshape(c.Hkv, -1)[:, :L])
    return out[0], out[2], out[3]


def _check(cache, lens, q, out, m=None, e=None, see_of=None, step=2.0 ** -33):
    """q, out [B][T][Hq][d], the last T tokens of each request; see_of(b, kvh): [T][L] (default:
    causal)."""
    B, T, Hq, d = q.shape
    scale, g = cache.case.scale, Hq // cache.case.Hkv
    for b in range(B):
        L = lens[b]
        K, V, vs = _held(cache, b, L)
        causal = torch.arange(L, device=DEV)[None] <= (L - T + torch.arange(T, device=DEV))[:, None]
        for h in range(Hq):
            k, v, s = K[h // g], V[h // g], vs[h // g]
            see = causal if see_of is None else see_of(b, h // g)
            x = (q[b, :, h].double() @ k.T * scale).masked_fill(~see, -np.inf)
            top = x.max(1).values
            none = torch.isinf(top)
            p = torch.exp(x - torch.where(none, 0.0, top)[:, None])
            total = p.sum(1)
            p = p / torch.where(none, 1.0, total)[:, None]
            want = p @ v
            mag = (q[b, :, h].double().abs() @ k.abs().T * abs(scale)).masked_fill(~see, 0.0)
            t = d * 2.0 ** -23 * mag.max(1).values + 2.0 ** -20 + (2 * -(-L // 16) + 2) * 2.0 ** -23
            most = (p * torch.where((v != 0).any(1), s, 0.0)).max(1).values
            codes = see.double() @ torch.where(s[:, None] > 0, v.abs() / s[:, None], 0.0)
            tol = t[:, None] * (p @ v.abs() + want.abs()) + step * most[:, None] * codes
            tol += 2.0 ** -140  # (steps of the smallest numbers)
            err = (out[b, :, h].double() - want).abs()
            bad = ~(err <= tol)
            assert not bad.any(), (b, h, bad.any(1).nonzero().flatten().tolist()[:8],
                                   (err / tol).nan_to_num(np.inf).max().item())
            if m is not None:
                ok = ~none
                assert (m[b, none, h] == -np.inf).all() and (e[b, none, h] == 0).all()
                assert ((m[b, :, h] - top).abs()[ok] <= (t + 2.0 ** -22 * top.abs())[ok]).all()
                assert ((e[b, :, h] / total - 1).abs()[ok] <= 2 * t[ok]).all()


def _prefill(cache, q, sparse=None):
    B, Tq, Hq, d = q.shape
    out = torch.full((B, Tq, Hq, d), float("nan"), device=DEV)
    m, e = (torch.full((B, Tq, Hq), float("nan"), device=DEV) for _ in range(2))
    dattn.dattn_prefill(cache.layout, cache.k_pool, cache.v_pool, q, cache.case.scale,
                        cache.seq_lens, out, m, e, sparse=sparse, dev_err=cache.dev_err)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    return out, m, e


SIZES = [10, 16, 22, 30, 100, float("inf")]
HEADS = [(4, 1, 128), (2, 1, 64), (3, 3, 64)]  # one, two and four query blocks to a CTA


def _grow(v, where, k):
    """Rows `where` of v times 2^k, or an infinity in each."""
    if np.isinf(k):
        v[where, :, 5] = float("inf")
    else:
        v[where] *= 2.0 ** k


@pytest.mark.parametrize("which", [slice(176, 192), [191], [165], slice(100, 120)])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_prefill_rows_that_do_not_see_a_large_value(Hq, Hkv, d, which):
    """A tile, a token, or a run across tiles whose V is 2^k times the others': the queries before it,
    in its own 64-token block and in blocks that a CTA holds beside it, keep their precision."""
    L, Tq, B = 192, 130, len(SIZES)
    case = W.Case("seen", B=B, Hq=Hq, Hkv=Hkv, d=d, P=32, lens=[0] * B, seed=3, reserve_tokens=L)
    cache = _cache(case)
    k, v = _rows((B, L, Hkv, d), 1), _rows((B, L, Hkv, d), 2)
    for b, size in enumerate(SIZES):
        _grow(v[b], which, size)
    cache.append(k, v)
    q = _rows((B, Tq, Hq, d), 3)
    out, m, e = _prefill(cache, q)
    _check(cache, [L] * B, q, out, m, e)


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_prefill_blocks_that_only_other_queries_keep(Hq, Hkv, d):
    """Block-sparse heads: odd query blocks keep key block 0, whose V is 2^k times larger."""
    L, Tq, B = 64 * 7, 64 * 5, len(SIZES)
    case = W.Case("kept", B=B, Hq=Hq, Hkv=Hkv, d=d, P=64, lens=[0] * B, seed=3, reserve_tokens=L)
    cache = _cache(case)
    k, v = _rows((B, L, Hkv, d), 4), _rows((B, L, Hkv, d), 5)
    for b, size in enumerate(SIZES):
        _grow(v[b], slice(0, 64), size)
    cache.append(k, v)
    lists = np.full((B, Hkv, 7, 3), -1, np.int32)
    for qb in range(7):
        lists[:, :, qb] = [qb, 0 if qb % 2 else 1, qb - 1 if qb > 1 else -1]
    sp = dattn.PrefillSparseConfig(torch.full((Hkv,), W.HEAD_RETRIEVAL, dtype=torch.int8, device=DEV),
                                   1, 1, torch.from_numpy(lists).to(DEV))
    q = _rows((B, Tq, Hq, d), 6)
    out, m, e = _prefill(cache, q, sp)
    key, pos = np.arange(L)[None], (L - Tq + np.arange(Tq))[:, None]

    def see_of(b, kvh):
        held = (lists[b, kvh][:, :, None] == np.arange(7)).any(1)
        return torch.from_numpy((key <= pos) & held[pos // 64, key // 64]).to(DEV)

    _check(cache, [L] * B, q, out, m, e, see_of)


@pytest.mark.parametrize("Tq,Hkv", [(1, 1), (70, 2), (70, 20)])
@pytest.mark.parametrize("drop", [20.0, 45.0, 200.0])
def test_prefill_of_large_values_that_weigh_little(Tq, Hkv, drop):
    """A visible block of large values whose keys score `drop` below the others: at 2^30 and e^-20 both
    count, at e^-200 only the small values do. Clusters of CTAs and CTAs by themselves."""
    d, L, B = 64, 64 * 75, 3
    case = W.Case("light", B=B, Hq=4 * Hkv, Hkv=Hkv, d=d, P=64, lens=[0] * B, seed=3,
                  reserve_tokens=L, scale=1.0)
    cache = _cache(case)
    k, v = _rows((B, L, Hkv, d), 7) * 0.125, _rows((B, L, Hkv, d), 8)
    k[..., 0] = 0.0
    for b, size in enumerate([12, 30, 100]):
        at = slice(64 * 40, 64 * 41 + 16)
        v[b, at] *= 2.0 ** size
        k[b, at, :, 0] = -drop / 2
    cache.append(k, v)
    q = _rows((B, Tq, 4 * Hkv, d), 9)
    q[..., 0] = 2.0
    out, m, e = _prefill(cache, q)
    _check(cache, [L] * B, q, out, m, e)


@pytest.mark.parametrize("Tq,Hkv", [(5, 1), (100, 2), (70, 20)])
@pytest.mark.parametrize("spread", [12, 40, 110])
def test_prefill_of_values_of_every_size(Tq, Hkv, spread):
    """Every tile's V has a size of its own, over enough key blocks for several emptyings of the
    accumulators; sharp scores, so that rows differ in which tiles count; zeros among them."""
    d, L = 64, 64 * 80 - 5
    case = W.Case("every", B=1, Hq=4 * Hkv, Hkv=Hkv, d=d, P=16, lens=[0], seed=3, reserve_tokens=L,
                  scale=0.5)
    cache = _cache(case)
    rng = np.random.default_rng(spread)
    k, v = _rows((1, L, Hkv, d), 10), _rows((1, L, Hkv, d), 11)
    size = np.exp2(rng.integers(-spread, spread + 1, size=-(-L // 16))).repeat(16)[:L]
    v *= torch.from_numpy(size).to(DEV)[None, :, None, None].to(torch.bfloat16)
    v[:, 320:352] = 0.0
    v[:, 1000:5000:7] = 0.0
    cache.append(k, v)
    q = _rows((1, Tq, 4 * Hkv, d), 12)
    out, m, e = _prefill(cache, q)
    _check(cache, [L], q, out, m, e)


def test_prefill_of_zero_values():
    """Values that are all zeros weigh in the sum as any others."""
    d, L, Tq = 128, 200, 90
    case = W.Case("zero", B=2, Hq=4, Hkv=1, d=d, P=16, lens=[0, 0], seed=3, reserve_tokens=L)
    cache = _cache(case)
    k, v = _rows((2, L, 1, d), 13), _rows((2, L, 1, d), 14)
    v[0] = 0.0
    v[1, :150] = 0.0
    cache.append(k, v)
    q = _rows((2, Tq, 4, d), 15)
    out, m, e = _prefill(cache, q)
    assert (out[0] == 0).all()
    _check(cache, [L, L], q, out, m, e)


@pytest.mark.parametrize("size", SIZES)
def test_prefill_after_a_taken_back_outlier(size):
    """An appended token is taken back (the length set back) and another one appended: its page keeps
    the larger scale and codes rounded to it; the pages before keep their weight."""
    d, L, Tq = 64, 84, 30
    case = W.Case("back", B=1, Hq=4, Hkv=1, d=d, P=16, lens=[0], seed=3, reserve_tokens=L + 8)
    cache = _cache(case)
    k, v = _rows((1, L, 1, d), 16), _rows((1, L, 1, d), 17)
    cache.append(k[:, :70].contiguous(), v[:, :70].contiguous())
    kx, vx = _rows((1, 3, 1, d), 18), _rows((1, 3, 1, d), 19)
    _grow(vx[0], slice(1, 2), size)
    cache.append(kx, vx)
    cache.seq_lens.fill_(70)
    cache.append(k[:, 70:].contiguous(), v[:, 70:].contiguous())
    q = _rows((1, Tq, 4, d), 20)
    out, m, e = _prefill(cache, q)
    _check(cache, [L], q, out, m, e)


# ---------------------------------------------------------------- decode
# A weight is right to 22 bits, or to 2^-40 of the largest of its warp where the tile's part of that
# cannot exceed 2^-22 of the sums so far: the t of 16 keys, 2^-23 and 2^-23, holds it for the products
# of a tile. (In the bound's terms 2^-28 for 2^-33, where V scales are within 2^12 of each other.)
DECODE = 2.0 ** -28


@pytest.mark.parametrize("size", SIZES)
def test_decode_after_a_taken_back_outlier(size):
    d, L = 64, 84
    case = W.Case("back", B=1, Hq=4, Hkv=1, d=d, P=16, lens=[0], seed=3, reserve_tokens=L + 8)
    cache = _cache(case)
    k, v = _rows((1, L, 1, d), 16), _rows((1, L, 1, d), 17)
    cache.append(k[:, :70].contiguous(), v[:, :70].contiguous())
    kx, vx = _rows((1, 3, 1, d), 18), _rows((1, 3, 1, d), 19)
    _grow(vx[0], slice(1, 2), size)
    cache.append(kx, vx)
    cache.seq_lens.fill_(70)
    cache.append(k[:, 70:].contiguous(), v[:, 70:].contiguous())
    q = _rows((1, 1, 4, d), 20)
    for splits in (0, 1):
        out = torch.empty(1, 4, d, device=DEV)
        cache.decode(q[:, 0].contiguous(), out, cache.workspace(num_splits=splits), num_splits=splits)
        torch.cuda.synchronize()
        _check(cache, [L], q, out[:, None], step=DECODE)


@pytest.mark.parametrize("T,g,splits", [(2, 4, 0), (8, 1, 0), (4, 2, 1), (3, 2, 7)])
def test_multi_query_decode_beside_a_large_value(T, g, splits):
    """The last of T new tokens has the large V: the queries before it do not see it."""
    d, L, B = 128, 1500, len(SIZES)
    case = W.Case("draft", B=B, Hq=2 * g, Hkv=2, d=d, P=16, lens=[0] * B, seed=3, reserve_tokens=L)
    cache = _cache(case)
    k, v = _rows((B, L, 2, d), 21), _rows((B, L, 2, d), 22)
    for b, size in enumerate(SIZES):
        _grow(v[b], [L - 1], size)
    cache.append(k, v)
    q = _rows((B, T, 2 * g, d), 23)
    out = torch.empty(B, T, 2 * g, d, device=DEV)
    m, e = torch.empty(B, T, 2 * g, device=DEV), torch.empty(B, T, 2 * g, device=DEV)
    cache.decode(q, out, cache.workspace(queries=T, num_splits=splits), m, e, num_splits=splits)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    _check(cache, [L] * B, q, out, m, e, step=DECODE)


@pytest.mark.parametrize("Hq,splits", [(2, 1), (16, 1), (16, 0)])
@pytest.mark.parametrize("drop", [20.0, 45.0, 200.0])
def test_decode_of_large_values_that_weigh_little(Hq, splits, drop):
    """A visible tile of large values whose keys score `drop` below the others, and taken in before
    them or after."""
    d, L, B = 128, 700, 6
    case = W.Case("dlight", B=B, Hq=Hq, Hkv=2, d=d, P=64, lens=[0] * B, seed=3, reserve_tokens=L,
                  scale=1.0)
    cache = _cache(case)
    k, v = _rows((B, L, 2, d), 24) * 0.125, _rows((B, L, 2, d), 25)
    k[..., 0] = 0.0
    for b in range(B):
        at = slice(0, 16) if b % 2 else slice(640, 660)
        v[b, at] *= 2.0 ** [12, 30, 100][b // 2]
        k[b, at, :, 0] = -drop / 2
    cache.append(k, v)
    q = _rows((B, 1, Hq, d), 26)
    q[..., 0] = 2.0
    out = torch.empty(B, Hq, d, device=DEV)
    m, e = torch.empty(B, Hq, device=DEV), torch.empty(B, Hq, device=DEV)
    cache.decode(q[:, 0].contiguous(), out, cache.workspace(num_splits=splits), m, e,
                 num_splits=splits)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    _check(cache, [L] * B, q, out[:, None], m[:, None], e[:, None], step=DECODE)


@pytest.mark.parametrize("T,Hq,Hkv,d,splits", [(1, 2, 2, 128, 1), (1, 16, 2, 128, 0), (2, 8, 2, 64, 1),
                                               (8, 2, 2, 128, 3)])
@pytest.mark.parametrize("every,size", [(5, 0.0), (1, 0.0), (5, 2.0 ** -30), (16, 2.0 ** -30)])
def test_heavy_tokens_without_values(T, Hq, Hkv, d, splits, every, size):
    """Every fifth token, one of each tile, or only the first (every = 1) scores 20 above the others and
    has a V of zeros or of 2^-30 of theirs: the others' small weights make the result."""
    L, B = 1500, 2
    case = W.Case("heavy", B=B, Hq=Hq, Hkv=Hkv, d=d, P=32, lens=[0] * B, seed=3, reserve_tokens=L,
                  scale=1.0)
    cache = _cache(case)
    k, v = _rows((B, L, Hkv, d), 31) * 0.125, _rows((B, L, Hkv, d), 32)
    k[..., 0] = 0.0
    heavy = slice(0, 1) if every == 1 else slice(0, L, every)
    k[:, heavy, :, 0] = 10.0
    v[:, heavy] *= size
    cache.append(k, v)
    q = _rows((B, T, Hq, d), 33)
    q[..., 0] = 2.0
    out = torch.empty(B, T, Hq, d, device=DEV)
    m, e = torch.empty(B, T, Hq, device=DEV), torch.empty(B, T, Hq, device=DEV)
    ws = cache.workspace(queries=T, num_splits=splits)
    if T == 1:
        cache.decode(q[:, 0].contiguous(), out, ws, m, e, num_splits=splits)
    else:
        cache.decode(q, out, ws, m, e, num_splits=splits)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    _check(cache, [L] * B, q, out, m, e, step=DECODE)
    out, m, e = _prefill(cache, q)
    _check(cache, [L] * B, q, out, m, e)
