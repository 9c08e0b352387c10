"""The cache read back (dattn_kv_read) against the codes' values in 64 bits."""
import numpy as np
import pytest
import torch

from _paged import FORMATS, Paged

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def dattn():
    import split_kv_decode_distattention_gb300 as dattn
    dattn.load_library()
    return dattn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


CASES = [
    # (lens, starts, counts, Hkv, d, P)
    ([1], None, [1], 1, 64, 16),
    ([300, 17, 64, 1], None, [300, 17, 64, 1], 2, 128, 16),
    ([300, 17, 64, 1], [33, 16, 0, 0], [200, 1, 0, 1], 3, 128, 32),
    ([500, 0, 900], [499, 0, 5], [1, 0, 895], 5, 64, 64),
    ([33] * 40, [7] * 40, [26] * 40, 4, 128, 256),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_rows_are_the_codes_values(dattn, fmt, case, dtype):
    lens, starts, counts, Hkv, d, P = CASES[case]
    pool = Paged(fmt, lens, Hkv, d, P, seed=case)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    ends = np.concatenate([[2], 2 + np.cumsum(counts)])  # two rows before the first request's
    N = int(ends[-1]) + 3                               # and three behind the last one's
    # k into a slice of a wider projection, v dense
    wide = torch.full((N, Hkv + 2, d), 9.0, dtype=dtype, device=DEV)
    k, v = wide[:, 1:1 + Hkv], torch.full((N, Hkv, d), 9.0, dtype=dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dattn.dattn_kv_read(lay, kp, vp, k, v, i32(ends.tolist()), i32(lens),
                        starts=None if starts is None else i32(starts), dev_err=err)
    assert int(err) == 0
    # fp32: code * scale rounded once (block scales and bf16 values are exact); bf16: rounded again
    for what, got in (("k", k), ("v", v)):
        g = got.double().cpu().numpy()
        assert (g[:2] == 9).all() and (g[ends[-1]:] == 9).all(), "rows of no request changed"
        for b in range(len(lens)):
            lo = 0 if starts is None else starts[b]
            ref = pool.rows(what, b, lo, lo + counts[b])
            x = g[ends[b]:ends[b + 1]]
            if fmt in ("bf16", "fp8-block"):
                assert np.array_equal(x, ref)  # bf16 numbers
            else:
                lim = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
                assert (np.abs(x - ref) <= lim * np.abs(ref) * (1 + 2.0 ** -20)).all()
    assert (wide[:, 0] == 9).all() and (wide[:, Hkv + 1:] == 9).all()


@pytest.mark.parametrize("fmt", ("bf16", "mixed"))
def test_one_of_k_and_v(dattn, fmt):
    pool = Paged(fmt, [70, 50], 2, 64, 16, seed=9)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    k, v, k1, v1 = (torch.empty(120, 2, 64, device=DEV) for _ in range(4))
    at = i32([0, 70, 120]), i32([70, 50])
    dattn.dattn_kv_read(lay, kp, vp, k, v, *at)
    dattn.dattn_kv_read(lay, kp, vp, k1, None, *at)
    dattn.dattn_kv_read(lay, kp, vp, None, v1, *at)
    assert torch.equal(k, k1) and torch.equal(v, v1)


def test_tokens_that_are_not_there_are_flagged_and_left(dattn):
    pool = Paged("fp8", [40, 40, 40, 40], 2, 64, 16, seed=4)
    pool.table[1, 1] = -1
    pool.table[2, 0] = pool.pages + 7
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    E = dattn.DEVERR

    def read(b, start, n):
        k, v = (torch.full((n, 2, 64), 9.0, device=DEV) for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ends = [0] * (b + 1) + [n] * (4 - b)
        dattn.dattn_kv_read(lay, kp, vp, k, v, i32(ends), i32([40] * 4),
                            starts=i32([start] * 4), dev_err=err)
        left = ((k == 9).all(-1).all(-1) & (v == 9).all(-1).all(-1)).tolist()
        return int(err), left

    assert read(0, 30, 10) == (0, [False] * 10)
    assert read(0, 35, 10) == (E["LEN_OOB"], [False] * 5 + [True] * 5)
    assert read(0, -2, 4) == (E["LEN_OOB"], [True] * 4)
    assert read(0, 2**31 - 1, 3) == (E["LEN_OOB"], [True] * 3)
    assert read(1, 14, 4) == (E["UNMAPPED_PAGE"], [False] * 2 + [True] * 2)
    assert read(2, 14, 4) == (E["PAGE_OOB"], [True] * 2 + [False] * 2)


def test_no_rows_is_nothing_to_read(dattn):
    pool = Paged("bf16", [40], 2, 64, 16, seed=4)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    none = torch.empty(0, 2, 64, device=DEV)
    dattn.dattn_kv_read(lay, kp, vp, none, none, i32([0, 0]), i32([40]))


def test_bounds_out_of_order_are_flagged(dattn):
    pool = Paged("bf16", [40, 40, 40], 2, 64, 16, seed=4)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    for ends in ([0, 30, 10, 40], [-5, 10, 20, 30], [0, 40, 80, 5]):
        k, v = (torch.full((60, 2, 64), 9.0, device=DEV) for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        dattn.dattn_kv_read(lay, kp, vp, k, v, i32(ends), i32([40] * 3), dev_err=err)
        torch.cuda.synchronize()
        assert int(err) & ~(dattn.DEVERR["CHUNK_OOB"] | dattn.DEVERR["LEN_OOB"]) == 0
        assert torch.isfinite(k).all()


def test_append_then_read(dattn):
    """What the append stored comes back: within half a code's step of what was appended."""
    Hkv, d, P, T = 2, 128, 16, 50
    for fmt in (dattn.KV_BF16, dattn.KV_FP8_E4M3, dattn.KV_INT4, dattn.KV_FP8_BLOCK):
        table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
        n = 8 * Hkv * P
        dt = torch.bfloat16 if fmt == dattn.KV_BF16 else torch.uint8
        width = d // 2 if fmt == dattn.KV_INT4 else d
        kp, vp = (torch.zeros(n * width, dtype=dt, device=DEV) for _ in range(2))
        sc = torch.zeros(max(dattn.kv_scale_floats(fmt, 8, Hkv, P), 4), device=DEV)
        lay = dattn.KVLayout(8, Hkv, d, P, table, fmt, sc)
        lens = i32([0, 0])
        g = torch.Generator(device=DEV).manual_seed(fmt)
        k, v = (torch.randn(2, T, Hkv, d, device=DEV, generator=g).to(torch.bfloat16)
                for _ in range(2))
        dattn.dattn_kv_append(lay, kp, vp, None, k, v, lens)
        ko, vo = (torch.empty(2 * T, Hkv, d, device=DEV) for _ in range(2))
        dattn.dattn_kv_read(lay, kp, vp, ko, vo, i32([0, T, 2 * T]), lens)
        for x, y in ((k, ko), (v, vo)):
            x, y = x.double(), y.view(2, T, Hkv, d).double()
            if fmt == dattn.KV_BF16:
                assert torch.equal(x, y)
                continue
            top = x.abs().amax(-1, keepdim=True)
            if fmt == dattn.KV_INT4:      # steps of top / 7
                lim = top / 14 * (1 + 2.0 ** -20)
            else:                         # 2^-4 of the value, and 2^-10 of a scale below 2^-6 of it
                if fmt == dattn.KV_FP8_BLOCK:
                    top = torch.full_like(top, float(x.abs().max()) * 2)
                lim = x.abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + top / 448 * 2.0 ** -10
            assert ((x - y).abs() <= lim).all()


def test_read_in_a_graph_follows_its_arguments(dattn):
    pool = Paged("fp8-block", [100, 60], 2, 64, 16, seed=6)
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    k, v = (torch.zeros(160, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ends, lens, starts = i32([0, 100, 160]), i32([100, 60]), i32([0, 0])
    dattn.dattn_kv_read(lay, kp, vp, k, v, ends, lens, starts=starts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dattn.dattn_kv_read(lay, kp, vp, k, v, ends, lens, starts=starts)
    k.zero_(); v.zero_()
    ends.copy_(i32([0, 10, 15])); starts.copy_(i32([90, 55]))
    graph.replay()
    ref = np.concatenate((pool.rows("v", 0, 90, 100), pool.rows("v", 1, 55, 60)))
    assert np.array_equal(v[:15].double().cpu().numpy(), ref)
    assert (v[15:] == 0).all()
