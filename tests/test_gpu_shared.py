"""The decode of a batch whose requests share prefixes (dattn_decode_shared) against attention over each
request's tokens in 64 bits."""
import numpy as np
import pytest
import torch

from _block_ref import attention
from _paged import Paged, bf16, check, weight_error

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def dattn():
    import split_kv_decode_distattention_gb300 as dattn
    dattn.load_library()
    return dattn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def queries(B, T, Hq, d, seed):
    return bf16(np.random.default_rng(seed).standard_normal((B, T, Hq, d))).to(DEV)


def check_all(pool, q, out, m, e, scale, what):
    B, T, Hq, d = q.shape
    g = Hq // pool.Hkv
    qn = q.double().cpu().numpy()
    for b in range(B):
        L = pool.lens[b]
        see = np.arange(L)[None] <= np.arange(L - T, L)[:, None]
        K, V = pool.rows("k", b), pool.rows("v", b)
        for h in range(Hq):
            ref, rm, re, bound, t = attention(qn[b, :, h], K[:, h // g], V[:, h // g], scale, see,
                                              weight_error("bf16"))
            check(out[b, :, h], None if m is None else m[b, :, h], None if e is None else e[b, :, h],
                  ref, bound, t, rm, re, f"{what} b={b} h={h} L={L}")


# (groups as (requests, prefix in the pages, prefix told), own tokens of every request, T, Hq, Hkv, d, P)
CASES = [
    # one group, rows of a tile and less; a prefix of one block, of less, of more
    ([(4, 64, 64)], [1, 5, 33, 100], 1, 8, 2, 128, 16),
    ([(4, 48, 48)], [1, 5, 33, 100], 1, 8, 2, 64, 16),
    ([(3, 1040, 1040)], [17, 2, 60], 2, 4, 2, 128, 16),
    # told less than the pages share, on no block or tile boundary
    ([(3, 1040, 1001)], [17, 2, 60], 2, 4, 2, 128, 16),
    ([(3, 512, 1)], [17, 2, 60], 1, 8, 8, 64, 64),
    # 129 and 257 rows of a KV head: one row behind a tile, and behind a CTA's two
    ([(43, 192, 192)], [1 + i % 7 for i in range(43)], 1, 3, 1, 64, 16),
    ([(33, 192, 192)], [8 + i % 7 for i in range(33)], 8, 1, 1, 128, 16),
    # ragged groups, one of a single request, one without a prefix, one without requests
    ([(5, 300, 288), (1, 700, 640), (0, 0, 500), (7, 0, 0), (20, 2000, 2000)],
     [3 + 5 * i for i in range(33)], 1, 8, 2, 128, 16),
    ([(9, 3000, 2944), (8, 700, 640)], [4 + i for i in range(17)], 4, 4, 2, 64, 128),
    # a long prefix: rows of several emptyings of the accumulators
    ([(2, 70000, 70000)], [40, 9], 1, 2, 1, 64, 64),
]


def build(fmt, groups, own, Hkv, d, P, seed):
    lens, shared, ends, told = [], [], [0], []
    for n, pages, prefix in groups:
        lo = ends[-1]
        lens += [pages + own[lo + i] for i in range(n)]
        shared.append((lo, lo + n, pages // P * P))
        ends.append(lo + n)
        told.append(min(prefix, pages // P * P) if n else prefix)
    return Paged(fmt, lens, Hkv, d, P, seed, shared=[s for s in shared if s[1] > s[0]]), ends, told


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(dattn, fmt, case):
    groups, own, T, Hq, Hkv, d, P = CASES[case]
    pool, ends, told = build(fmt, groups, own, Hkv, d, P, case)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    B = len(pool.lens)
    q = queries(B, T, Hq, d, case + 30)
    ws = dattn.SharedWorkspace(B, T, Hq, Hkv, d)
    err = i32([0])
    scale = d ** -0.5
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((B + 1, T, Hq, d), 9.0, dtype=dtype, device=DEV)
        m, e = (torch.full((B, T, Hq), 9.0, device=DEV) for _ in range(2))
        dattn.dattn_decode_shared(lay, kp, vp, q, scale, i32(pool.lens), i32(ends), i32(told), out, ws,
                                  m, e, dev_err=err)
        assert int(err) == 0 and (out[B] == 9).all()
        check_all(pool, q, out, m, e, scale, f"{fmt} {dtype}")


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_requests_shorter_than_the_prefix_and_outside_of_groups(dattn, fmt):
    Hq, Hkv, d, P, T = 8, 2, 128, 16, 2
    lens = [500, 700, 16, 1, 0, 650, 300, 90]
    pool = Paged(fmt, lens, Hkv, d, P, seed=1, shared=[(1, 6, 640)])
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(8, T, Hq, d, 2)
    ws = dattn.SharedWorkspace(8, T, Hq, Hkv, d)
    out = torch.empty(8, T, Hq, d, device=DEV)
    m, e = (torch.empty(8, T, Hq, device=DEV) for _ in range(2))
    err = i32([0])
    dattn.dattn_decode_shared(lay, kp, vp, q, 0.1, i32(lens), i32([1, 6]), i32([640]), out, ws, m, e,
                              dev_err=err)
    assert int(err) == 0
    check_all(pool, q, out, m, e, 0.1, fmt)
    assert (out[4] == 0).all()


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_one_request_far_above_the_others_and_a_negative_scale(dattn, fmt):
    """Rows whose maxima lie 1000 apart, and climb along the prefix."""
    Hq, Hkv, d, P = 4, 1, 64, 16
    lens = [1000, 990, 970]
    pool = Paged(fmt, lens, Hkv, d, P, seed=3, shared=[(0, 3, 960)])
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(3, 1, Hq, d, 4)
    q[1] *= 64
    ws = dattn.SharedWorkspace(3, 1, Hq, Hkv, d)
    out = torch.empty(3, 1, Hq, d, device=DEV)
    for scale in (0.3, -0.3):
        dattn.dattn_decode_shared(lay, kp, vp, q, scale, i32(lens), i32([0, 3]), i32([960]), out, ws)
        check_all(pool, q, out, None, None, scale, f"{fmt} {scale}")


def test_bounds_out_of_order_are_flagged_and_every_request_attended(dattn):
    Hq, Hkv, d, P = 4, 2, 64, 16
    lens = [100, 90, 80]
    pool = Paged("bf16", lens, Hkv, d, P, seed=3, shared=[(0, 3, 64)])
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(3, 1, Hq, d, 4)
    ws = dattn.SharedWorkspace(3, 1, Hq, Hkv, d)
    for ends in ([0, 2, 1], [0, 2, 4], [-1, 2, 3], [2**31 - 1, 0, 3]):
        err = i32([0])
        out = torch.empty(3, 1, Hq, d, device=DEV)
        dattn.dattn_decode_shared(lay, kp, vp, q, 0.1, i32(lens), i32(ends), i32([64, 64]), out, ws,
                                  dev_err=err)
        assert int(err) == dattn.DEVERR["CHUNK_OOB"]
        check_all(pool, q, out, None, None, 0.1, str(ends))


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_bad_pages_of_the_prefix_are_flagged_and_left_out(dattn, fmt):
    Hq, Hkv, d, P = 4, 2, 64, 16
    lens = [200, 200]
    pool = Paged(fmt, lens, Hkv, d, P, seed=3, shared=[(0, 2, 160)])
    q = queries(2, 1, Hq, d, 4)
    ws = dattn.SharedWorkspace(2, 1, Hq, Hkv, d)
    E = dattn.DEVERR
    want = E["UNMAPPED_PAGE"] | E["PAGE_OOB"]
    K, V = ([pool.rows(w, b) for b in range(2)] for w in "kv")
    pool.table[:, 2], pool.table[:, 5] = -1, pool.pages
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    err = i32([0])
    out = torch.empty(2, 1, Hq, d, device=DEV)
    dattn.dattn_decode_shared(lay, kp, vp, q, 0.1, i32(lens), i32([0, 2]), i32([150]), out, ws,
                              dev_err=err)
    assert int(err) == want
    see = np.ones((1, 200), bool)
    see[:, 32:48] = see[:, 80:96] = False
    qn = q.double().cpu().numpy()
    for b in range(2):
        for h in range(Hq):
            ref, _, _, bound, _ = attention(qn[b, :, h], K[b][:, h // 2], V[b][:, h // 2], 0.1, see,
                                            weight_error("bf16"))
            check(out[b, :, h], None, None, ref, bound, 0, 0, 0, f"{fmt} b={b} h={h}")


def test_without_groups_it_is_the_multi_query_decode(dattn):
    lens = [300, 5]
    pool = Paged("fp8-block", lens, 2, 64, 16, seed=3)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(2, 2, 4, 64, 4)
    a, b = (torch.empty(2, 2, 4, 64, device=DEV) for _ in range(2))
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    dattn.dattn_decode_shared(lay, kp, vp, q, 0.1, i32(lens), i32([0]), none, a,
                              dattn.SharedWorkspace(2, 2, 4, 2, 64))
    dattn.dattn_decode_multi(lay, kp, vp, q, 0.1, i32(lens), b, dattn.Workspace(2, 8, 2, 64))
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_in_a_graph_and_twice_alike(dattn, fmt):
    """Replayed with other lengths, groups and prefixes; a second run gives the same bits."""
    Hq, Hkv, d, P = 8, 2, 128, 16
    lens = [900, 850, 840, 333]
    pool = Paged(fmt, lens, Hkv, d, P, seed=3, shared=[(0, 3, 800)])
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(4, 1, Hq, d, 4)
    ws = dattn.SharedWorkspace(4, 1, Hq, Hkv, d)
    L, ends, told = i32(lens), i32([0, 3, 4]), i32([800, 0])
    out, want = (torch.empty(4, 1, Hq, d, device=DEV) for _ in range(2))

    def call(to):
        dattn.dattn_decode_shared(lay, kp, vp, q, 0.1, L, ends, told, to, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for lens2, ends2, told2 in ((lens, [0, 3, 4], [800, 0]), ([810, 5, 840, 1], [0, 2, 3], [640, 100]),
                                (lens, [0, 0, 0], [800, 800]), (lens, [0, 3, 4], [800, 333])):
        L.copy_(i32(lens2)); ends.copy_(i32(ends2)); told.copy_(i32(told2))
        graph.replay()
        call(want)
        assert torch.equal(out, want)
        pool.lens = lens2
        check_all(pool, q, out, None, None, 0.1, f"{fmt} {ends2}")


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
@pytest.mark.parametrize("B", (3, 40))
def test_prefix_whose_pieces_are_joined_in_the_workspace(dattn, fmt, B):
    """1.4M tokens of prefix, so that a CTA's run is longer than what stays in its accumulators, for one
    tile of rows and for two. The prefix's pages repeat: a key counts as often as its page does."""
    Hq, Hkv, d, P, pages, reps = 4, 1, 64, 256, 4, 1370
    n = pages * reps
    base = Paged(fmt, [pages * P + P], Hkv, d, P, seed=13, spare=0)
    phys = base.table[0, :pages + 1]
    table = np.tile(phys[:pages], reps)[None].repeat(B, 0)
    table = np.concatenate((table, np.full((B, 1), phys[pages], np.int32)), 1).astype(np.int32)
    own = [1 + 5 * b for b in range(B)]  # of the last page, the same rows for all
    lens = [n * P + x for x in own]
    kp, vp = base.pools()
    sc = None if base.kv_scale is None else base.kv_scale.to(DEV)
    lay = dattn.KVLayout(base.pages, Hkv, d, P, torch.from_numpy(table).to(DEV),
                         0 if fmt == "bf16" else dattn.KV_FP8_BLOCK, sc)
    q = queries(B, 1, Hq, d, 14)
    ws = dattn.SharedWorkspace(B, 1, Hq, Hkv, d)
    err = i32([0])
    out, again = (torch.empty(B, 1, Hq, d, device=DEV) for _ in range(2))
    for to in (out, again):
        dattn.dattn_decode_shared(lay, kp, vp, q, 0.125, i32(lens), i32([0, B]), i32([n * P - 77]), to,
                                  ws, dev_err=err)
    assert int(err) == 0 and torch.equal(out, again)
    K, V = base.rows("k", 0)[:, 0], base.rows("v", 0)[:, 0]
    qn = q.double().cpu().numpy()
    for b in (0, 1, B - 1):
        L = pages * P + own[b]
        count = np.where(np.arange(L) < pages * P, reps, 1)
        for h in range(Hq):
            s = K[:L] @ qn[b, 0, h] * 0.125
            w = count * np.exp(s - s.max())
            ref = w @ V[:L] / w.sum()
            mag = np.abs(K[:L]) @ np.abs(qn[b, 0, h]) * 0.125
            # logits and weights as in attention(); sums of up to 64 blocks of 8 products, then of up to
            # 200 partials: each addition at most 2^-23 off
            t = d * 2.0 ** -23 * mag.max() + weight_error("bf16") + (64 * 8 + 200) * 2.0 ** -23
            check(out[b, :, h], None, None, ref[None], np.array([2 * t * np.abs(V[:L]).max()]), 0, 0, 0,
                  f"{fmt} b={b} h={h}")
