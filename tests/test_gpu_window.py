"""The sliding window with first tokens that stay visible (dattn_decode_window, dattn_prefill_window)
against its definition in 64 bits: the query at position p sees the keys i <= p with i > p - window or
i < sinks."""
import numpy as np
import pytest
import torch

from _block_ref import attention
from _paged import FORMATS, Paged, bf16, check, weight_error

pytestmark = pytest.mark.gpu

DEV = "cuda"
OVER = 1 << 30


@pytest.fixture(scope="module")
def dattn():
    import split_kv_decode_distattention_gb300 as dattn
    dattn.load_library()
    return dattn


def sees(L, T, window, sinks):
    """[T][L]: which keys the last T tokens see."""
    p = np.arange(L - T, L)[:, None]
    i = np.arange(L)[None]
    return (i <= p) & ((i > p - window) | (i < sinks))


def check_all(pool, q, out, m, e, scale, window, sinks, what):
    B, T, Hq, d = q.shape
    g = Hq // pool.Hkv
    qn = q.double().cpu().numpy()
    for b in range(B):
        L = pool.lens[b]
        see = sees(L, T, window, sinks)
        K, V = pool.rows("k", b), pool.rows("v", b)
        for h in range(Hq):
            ref, rm, re, bound, t = attention(qn[b, :, h], K[:, h // g], V[:, h // g], scale, see,
                                              weight_error(pool.fmt))
            check(out[b, :, h], None if m is None else m[b, :, h], None if e is None else e[b, :, h],
                  ref, bound, t, rm, re, f"{what} b={b} h={h} L={L}")


def queries(B, T, Hq, d, seed):
    return bf16(np.random.default_rng(seed).standard_normal((B, T, Hq, d))).to(DEV)


STEPS = [
    # (lens, T, Hq, Hkv, d, P, window, sinks)
    ([1, 5, 16, 17, 40, 0], 1, 4, 4, 128, 16, 7, 2),
    ([2000, 33, 515], 2, 8, 2, 128, 16, 100, 4),       # windows on no tile boundary
    ([2000, 33, 515], 2, 8, 2, 128, 64, 96, 16),       # and on one
    ([3, 1, 8, 700, 129], 8, 2, 2, 64, 16, 1, 0),      # a window of the token itself, lengths below T
    ([3, 1, 8, 700, 129], 8, 2, 2, 64, 16, 3, 1),
    ([900, 64], 4, 4, 2, 64, 32, OVER, 5),             # no window: all tokens
    ([900, 64], 3, 4, 2, 128, 32, 20, OVER),           # all tokens are first tokens
    ([1500, 70, 90], 1, 16, 2, 128, 128, 64, 17),      # sinks that end inside a tile; g = 8
    ([300, 301, 302, 303, 304, 305], 4, 6, 3, 64, 16, 13, 3),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_step_against_the_definition(dattn, fmt, case):
    lens, T, Hq, Hkv, d, P, window, sinks = STEPS[case]
    pool = Paged(fmt, lens, Hkv, d, P, seed=case)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    B = len(lens)
    q = queries(B, T, Hq, d, case + 50)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = dattn.Workspace(B, T * Hq, Hkv, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    scale = d ** -0.5
    for dtype, splits in ((torch.float32, 0), (torch.bfloat16, 5)):
        if splits:
            ws = dattn.Workspace(B, T * Hq, Hkv, d, num_splits=splits)
        out = torch.full((B, T, Hq, d), 9.0, dtype=dtype, device=DEV)
        m, e = (torch.full((B, T, Hq), 9.0, device=DEV) for _ in range(2))
        dattn.dattn_decode_window(lay, kp, vp, q, scale, L, window, sinks, out, ws, m, e,
                                  num_splits=splits, dev_err=err)
        assert int(err) == 0
        # (a query before the first token sees nothing: L < T)
        check_all(pool, q, out, m, e, scale, window, sinks, f"{fmt} splits={splits}")


@pytest.mark.parametrize("fmt", FORMATS)
def test_step_without_a_window_is_the_multi_query_decode(dattn, fmt):
    lens, T, Hq, Hkv, d = [1003, 17, 250], 2, 8, 2, 128
    pool = Paged(fmt, lens, Hkv, d, 16, seed=3)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(3, T, Hq, d, 4)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = dattn.Workspace(3, T * Hq, Hkv, d)
    a, b = (torch.empty(3, T, Hq, d, device=DEV) for _ in range(2))
    dattn.dattn_decode_multi(lay, kp, vp, q, 0.1, L, a, ws, num_splits=3)
    dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 5000, 0, b, ws, num_splits=3)
    assert torch.equal(a, b)


def test_step_of_one_token_is_what_a_streaming_head_attends(dattn):
    lens, Hq, Hkv, d = [1003, 17, 250, 0], 8, 2, 128
    pool = Paged("fp8", lens, Hkv, d, 16, seed=3)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(4, 1, Hq, d, 4)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = dattn.Workspace(4, Hq, Hkv, d)
    kind = torch.full((Hkv,), dattn.HEAD_STREAMING, dtype=torch.int8, device=DEV)
    a, b = (torch.empty(4, 1, Hq, d, device=DEV) for _ in range(2))
    dattn.dattn_decode(lay, kp, vp, q[:, 0], 0.1, L, a, ws,
                       sparse=dattn.SparseConfig(kind, 4, 33, 0, None))
    dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 33, 4, b, ws)
    # the same keys, split and summed in another order (fp32 sums of weights within 2^-22)
    assert (a - b).abs().max() < 1e-4


def test_step_flags_bad_lengths_and_pages(dattn):
    pool = Paged("bf16", [100, 100, 100], 2, 64, 16, seed=1)
    pool.table[1, 6] = -1
    pool.table[2, 5] = pool.pages
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(3, 1, 4, 64, 1)
    L = torch.tensor([-3, 100, 100], dtype=torch.int32, device=DEV)
    ws = dattn.Workspace(3, 4, 2, 64)
    out = torch.full((3, 1, 4, 64), 9.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 40, 0, out, ws, dev_err=err)
    E = dattn.DEVERR
    assert int(err) == E["LEN_OOB"] | E["UNMAPPED_PAGE"] | E["PAGE_OOB"]
    assert (out[0] == 0).all() and torch.isfinite(out).all()


def test_step_does_not_look_at_pages_that_the_window_left(dattn):
    """Pages behind the window may be unmapped (given back): nothing is flagged."""
    pool = Paged("fp8", [1000], 2, 64, 16, seed=2)
    free = pool.table.copy()
    free[0, 1:(1000 - 200) // 16] = -1  # all but the sinks' page and the window's
    q = queries(1, 2, 4, 64, 7)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    L = torch.tensor([1000], dtype=torch.int32, device=DEV)
    ws = dattn.Workspace(1, 8, 2, 64)
    a, b = (torch.empty(1, 2, 4, 64, device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 190, 5, a, ws)
    pool.table = free
    dattn.dattn_decode_window(pool.layout(dattn), kp, vp, q, 0.1, L, 190, 5, b, ws, dev_err=err)
    assert int(err) == 0 and torch.equal(a, b)


def test_step_in_a_graph_follows_the_lengths(dattn):
    pool = Paged("int4", [400, 90], 2, 128, 16, seed=5)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(2, 2, 4, 128, 8)
    L = torch.tensor([400, 90], dtype=torch.int32, device=DEV)
    ws = dattn.Workspace(2, 8, 2, 128)
    out, want = (torch.empty(2, 2, 4, 128, device=DEV) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 50, 4, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 50, 4, out, ws)
    for lens in ([400, 90], [33, 2], [399, 60]):
        L.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 50, 4, want, ws)
        assert torch.equal(out, want)


# ---- the prefill

CHUNKS = [
    # (lens, Tq, Hq, Hkv, d, P, window, sinks)
    ([70, 200, 641], 64, 4, 2, 128, 16, 100, 4),      # even groups: two heads to a tile
    ([70, 200, 641], 37, 4, 2, 128, 16, 64, 0),       # a window of one block
    ([130, 333], 130, 3, 3, 64, 32, 1, 0),            # the token itself alone; odd groups
    ([130, 333], 130, 3, 1, 64, 16, 1, 1),
    ([600, 601, 700], 129, 8, 2, 128, 64, 65, 64),    # sinks of one block; g = 4
    ([600, 601, 700], 129, 5, 1, 128, 64, 63, 65),
    ([1030, 900], 900, 8, 1, 64, 16, 200, 130),       # g = 8; sinks past two blocks
    ([500], 300, 4, 2, 128, 16, OVER, 3),             # no window
    ([500], 300, 4, 2, 128, 16, 5, OVER),             # all tokens are first tokens
    ([3000], 1, 8, 2, 128, 128, 777, 10),             # one token
    ([4200], 70, 4, 4, 64, 16, 3000, 5),              # more than 32 blocks seen by a row
    ([500, 333], 200, 7, 1, 128, 96, 150, 20),        # pages of 96 and 48 tokens; g = 7 and 6
    ([500, 333], 200, 12, 2, 64, 48, 150, 20),
]


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunk_against_the_definition(dattn, fmt, case):
    lens, T, Hq, Hkv, d, P, window, sinks = CHUNKS[case]
    pool = Paged(fmt, lens, Hkv, d, P, seed=case)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    B = len(lens)
    q = queries(B, T, Hq, d, case + 150)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((B + 1, T, Hq, d), 9.0, dtype=dtype, device=DEV)
        m, e = (torch.full((B, T, Hq), 9.0, device=DEV) for _ in range(2))
        dattn.dattn_prefill_window(lay, kp, vp, q, d ** -0.5, L, window, sinks, out, m, e,
                                   dev_err=err)
        assert int(err) == 0 and (out[B] == 9).all()
        check_all(pool, q, out, m, e, d ** -0.5, window, sinks, f"{fmt} {dtype}")


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_chunk_without_a_window_is_the_causal_prefill(dattn, fmt):
    pool = Paged(fmt, [700, 400], 2, 128, 16, seed=3)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(2, 300, 8, 128, 4)
    L = torch.tensor([700, 400], dtype=torch.int32, device=DEV)
    a, b = (torch.empty(2, 300, 8, 128, device=DEV) for _ in range(2))
    dattn.dattn_prefill(lay, kp, vp, q, 0.1, L, a)
    dattn.dattn_prefill_window(lay, kp, vp, q, 0.1, L, 700, 0, b)
    # Two kernels that cut and sum the same keys differently: each is within the bound of the exact
    # result, so the two are within twice the bound of each other.
    for r, n in enumerate((700, 400)):
        K, V = pool.rows("k", r), pool.rows("v", r)
        for h in range(8):
            _, _, _, bound, _ = attention(q[r, :, h].double().cpu().numpy(), K[:, h // 4], V[:, h // 4],
                                          0.1, sees(n, 300, 700, 0), weight_error("bf16"))
            d = (a[r, :, h] - b[r, :, h]).abs().amax(-1).double().cpu().numpy()
            assert (d <= 2 * bound).all()


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_chunk_of_a_few_tokens_is_the_step(dattn, fmt):
    pool = Paged(fmt, [700, 93], 2, 128, 16, seed=8)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(2, 4, 4, 128, 9)
    L = torch.tensor([700, 93], dtype=torch.int32, device=DEV)
    a, b = (torch.empty(2, 4, 4, 128, device=DEV) for _ in range(2))
    dattn.dattn_prefill_window(lay, kp, vp, q, 0.1, L, 100, 7, a)
    dattn.dattn_decode_window(lay, kp, vp, q, 0.1, L, 100, 7, b, dattn.Workspace(2, 16, 2, 128))
    # weights within 2^-17 of theirs in both, values below 2^3
    assert (a - b).abs().max() < 4 * 2.0 ** -17 * 8


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
def test_chunk_behind_a_long_context_reads_its_window_alone(dattn, fmt):
    """70K tokens whose pages behind the sinks and before the window are unmapped."""
    Hkv, d, P, T, W, S = 1, 64, 64, 90, 150, 70
    lens = [70_001]
    keep = Paged(fmt, [S + P + W + T + 2 * P], Hkv, d, P, seed=10)  # a pool of the pages in use
    n = lens[0] // P + 1
    first = (lens[0] - T - W + 1) // P
    table = np.full((1, n), -1, np.int32)
    used = [0, 1] + list(range(first, n))
    table[0, used] = keep.table[0, :len(used)]
    q = queries(1, T, 2, d, 11)
    keep.k, keep.v = np.nan_to_num(keep.k), np.nan_to_num(keep.v)
    near = Paged.__new__(Paged)
    near.__dict__.update(keep.__dict__)
    near.table, near.lens = table, lens
    lay, (kp, vp) = near.layout(dattn), near.pools()
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty(1, T, 2, d, device=DEV)
    dattn.dattn_prefill_window(lay, kp, vp, q, 0.2, L, W, S, out, dev_err=err)
    assert int(err) == 0
    see = sees(lens[0], T, W, S)
    seen = see.any(0)
    tok = np.flatnonzero(seen)
    K, V = (x[table[0][tok // P], 0, tok % P] for x in (near.k, near.v))
    for h in range(2):
        ref, _, _, bound, _ = attention(q[0, :, h].double().cpu().numpy(), K, V, 0.2, see[:, seen],
                                        weight_error(fmt))
        check(out[0, :, h], None, None, ref, bound, 0, 0, 0, f"{fmt} h={h}")


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
@pytest.mark.parametrize("P", (16, 32, 48, 64))
def test_chunk_does_not_look_at_pages_that_its_windows_left(dattn, fmt, P):
    """Pages without a token that some query sees may be given back, inside a block of 64 too."""
    lens, T, W, S = [1000, 431], 90, 190, 5
    pool = Paged(fmt, lens, 2, 64, P, seed=12)
    q = queries(2, T, 4, 64, 7)
    (kp, vp), L = pool.pools(), torch.tensor(lens, dtype=torch.int32, device=DEV)
    a, b = (torch.empty(2, T, 4, 64, device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dattn.dattn_prefill_window(pool.layout(dattn), kp, vp, q, 0.1, L, W, S, a)
    pool.table = pool.table.copy()
    for r, n in enumerate(lens):
        first = n - T - W + 1  # the first key of the first query's window
        pool.table[r, -(-S // P):first // P] = -1
    dattn.dattn_prefill_window(pool.layout(dattn), kp, vp, q, 0.1, L, W, S, b, dev_err=err)
    assert int(err) == 0 and torch.equal(a, b)


def test_chunk_flags_a_length_below_it(dattn):
    pool = Paged("bf16", [100, 100], 2, 64, 16, seed=1)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(2, 50, 4, 64, 1)
    out = torch.full((2, 50, 4, 64), 9.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dattn.dattn_prefill_window(lay, kp, vp, q, 0.1, torch.tensor([49, 100], dtype=torch.int32,
                                                                 device=DEV), 20, 0, out, dev_err=err)
    assert int(err) == dattn.DEVERR["LEN_OOB"]
    assert (out[0] == 9).all() and (out[1] != 9).all()


@pytest.mark.parametrize("fmt", ("bf16", "fp8-block"))
@pytest.mark.parametrize("g", (4, 3))
def test_chunk_of_many_tiles_for_each_sm(dattn, fmt, g):
    """Many more tiles than SMs: a CTA goes from one to the next, and its last ones are of another kind."""
    T, Hkv, d, W, S = 3000, 8, 64, 130, 5
    lens = [3010, 3000, 4100]
    pool = Paged(fmt, lens, Hkv, d, 64, seed=21)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    q = queries(3, T, g * Hkv, d, 22)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.empty(3, T, g * Hkv, d, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dattn.dattn_prefill_window(lay, kp, vp, q, 0.125, L, W, S, out, dev_err=err)
    assert int(err) == 0
    for b in range(3):
        for h in (0, g * Hkv - 1, 11):
            ref, _, _, bound, _ = attention(q[b, :, h].double().cpu().numpy(),
                                            pool.rows("k", b)[:, h // g], pool.rows("v", b)[:, h // g],
                                            0.125, sees(lens[b], T, W, S), weight_error("bf16"))
            check(out[b, :, h], None, None, ref, bound, 0, 0, 0, f"{fmt} g={g} b={b} h={h}")


def test_every_code_of_the_block_scaled_pool_comes_through_exactly(dattn):
    """One key with weight 1: the output is its V row. All codes but NaN, scales from 2^-100 to 2^100;
    a NaN code gives NaN in its channel."""
    d, P = 128, 16
    codes = torch.arange(256, dtype=torch.uint8)
    for k in (-100, -9, 0, 20, 100):
        kp = torch.zeros(2, 1, P, d, dtype=torch.uint8)
        vp = torch.zeros(2, 1, P, d, dtype=torch.uint8)
        vp[:, 0, 0] = codes.view(2, d)
        sc = torch.tensor([1.0, 2.0 ** k, 1.0, 2.0 ** k], device=DEV)
        lay = dattn.KVLayout(2, 1, d, P, torch.tensor([[0], [1]], dtype=torch.int32, device=DEV),
                             dattn.KV_FP8_BLOCK, sc)
        q = torch.zeros(2, 1, 1, d, dtype=torch.bfloat16, device=DEV)
        out = torch.empty(2, 1, 1, d, device=DEV)
        dattn.dattn_prefill_window(lay, kp.to(DEV), vp.to(DEV), q, 1.0,
                                   torch.ones(2, dtype=torch.int32, device=DEV), 5, 0, out)
        ref = codes.view(torch.float8_e4m3fn).double() * 2.0 ** k
        got = out.double().cpu().view(-1)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))
