"""The rotation and the rotating append on the GPU.

dattn_rope is compared with a 64-bit rotation whose angles are reduced exactly. Error of one
result, in units of (|x_a| + |x_b|) A: the angle (2^-32 of a turn, its fp32 value
of at most an eighth of a turn scaled to radians: 2^-24 of pi/4 three times) under 1.5e-7, the
polynomials' roundings and omitted terms under 1e-7, the product with A and the two products and
the sum 2^-24 each, 2.4e-7 and less: under 2^-21 = 4.8e-7 together, as the errors of a pair's sine
and cosine meet |x_a| and |x_b| once each. To that comes half a step of the result's type.

dattn_rope_append is compared bit for bit with dattn_rope followed by dattn_kv_append.
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
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _rand(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _positions(n, seed, far):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-far, far + 1, (n,), generator=g, device=DEV).to(torch.int32)


def _check_rope(x, y, pos, rot, inverse):
    n = rot.rot_dim // 2
    x64 = x.double().cpu().numpy()
    want = ref.rotate(x64, pos.cpu().numpy(), rot.inv_freq, bool(rot.c.interleaved), inverse,
                      rot.c.amplitude)
    tol = HALF[x.dtype] * np.abs(want) + 2.0 ** -21 * ref.partner_sum(
        x64, n, bool(rot.c.interleaved)) * abs(rot.c.amplitude)
    tol[..., 2 * n:] = 0  # unrotated channels are copied
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 96), (128, 48), (128, 16), (64, 64), (64, 32),
                                   (64, 48), (64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_against_64_bits(dtype, d, rot, interleaved):
    r = dattn.Rotation(rot, interleaved=interleaved, base=500000.0, amplitude=1.25)
    for N, H, far in ((1, 1, 1 << 20), (16, 9, 3), (37, 5, 1 << 24)):
        x = _rand((N, H, d), N + d + rot, dtype)
        pos = _positions(N, N, far)
        y = torch.full_like(x, float("nan"))
        inverse = N == 37
        dattn.dattn_rope(r, x, y, pos, inverse=inverse)
        _check_rope(x, y, pos, r, inverse)


def test_rope_at_the_ends_of_the_positions():
    """Positions 0, +-1 and the int32 limits; fast and slow frequencies, one above a turn."""
    f = [1.0, 6.9, 0.3, 1e-3, 1e-9, 0.0, 2.5, 1e-5]
    r = dattn.Rotation(16, inv_freq=f)
    pos = torch.tensor([0, 1, -1, 2 ** 30, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    x = _rand((6, 3, 64), 1, torch.float32)
    y = torch.empty_like(x)
    dattn.dattn_rope(r, x, y, pos)
    torch.testing.assert_close(y[0], x[0], rtol=0, atol=0)  # position 0 turns nothing
    want = ref.rotate(x.double().cpu().numpy(), pos.tolist(), r.inv_freq)
    # the double quotient f / 2 pi is off by 2^-53 f turns: at 2^31, 2^-22 f turns
    tol = 2.0 ** -24 * np.abs(want) + (2.0 ** -21 + 2.0 ** -22 * 2 * np.pi * max(f)) * \
        ref.partner_sum(x.double().cpu().numpy(), 8)
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


def test_rope_takes_slices_and_works_in_place():
    r = dattn.Rotation(64)
    B, T, H, d = 3, 21, 6, 128
    qkv = _rand((B, T, 10, d), 2)
    x = qkv[:, :, 2:2 + H]
    pos = _positions(B * T, 3, 5000).view(B, T)
    y = torch.empty(B, T, H, d, dtype=torch.bfloat16, device=DEV)
    dattn.dattn_rope(r, x, y, pos)
    whole = x.contiguous()
    _check_rope(whole.view(B * T, H, d), y.view(B * T, H, d), pos.view(-1), r, False)
    before = qkv.clone()
    dattn.dattn_rope(r, x, x, pos)  # in place, in the fused projection
    assert torch.equal(x, y)
    assert torch.equal(qkv[:, :, :2], before[:, :, :2]) and torch.equal(qkv[:, :, 8:],
                                                                       before[:, :, 8:])
    empty = torch.empty(0, H, d, dtype=torch.bfloat16, device=DEV)
    dattn.dattn_rope(r, empty, empty, pos.view(-1))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """inverse=True is the gradient: against differences (the map is linear, so a step of 1 has no
    truncation error) and against the 64-bit transpose."""
    r = dattn.Rotation(96, interleaved=interleaved, amplitude=0.75)
    N, H, d = 19, 3, 128
    x, dx, dy = (_rand((N, H, d), s, torch.float32) for s in (1, 2, 3))
    pos = _positions(N, 4, 1 << 20)
    f = lambda v: dattn.dattn_rope(r, v, v, pos) or v.double()  # noqa: E731
    g = dy.clone()
    dattn.dattn_rope(r, g, g, pos, inverse=True)
    _check_rope(dy, g, pos, r, True)
    hi, lo = x + dx, x - dx
    step = (hi - lo).double() / 2  # the step taken, after rounding
    diff = (f(hi.clone()) - f(lo.clone())) / 2
    lhs, rhs = (diff * dy).sum().item(), (step * g).sum().item()
    mag = sum(ref.partner_sum(t.double().cpu().numpy(), 48, interleaved) +
              np.abs(t.double().cpu().numpy()) for t in (hi, lo))
    tol = 2.0 ** -20 * (mag * np.abs(dy.double().cpu().numpy())).sum()
    tol += 2.0 ** -20 * ((ref.partner_sum(dy.double().cpu().numpy(), 48, interleaved) +
                          dy.abs().double().cpu().numpy()) *
                         step.abs().cpu().numpy()).sum()
    assert abs(lhs - rhs) <= tol


def test_rope_on_another_stream_and_in_a_graph():
    r = dattn.Rotation(128)
    x = _rand((130, 8, 128), 5)
    pos = _positions(130, 6, 9000)
    want = torch.empty_like(x)
    dattn.dattn_rope(r, x, want, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.zeros_like(x)
    dattn.dattn_rope(r, x, y, pos, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    z = torch.zeros_like(x)
    with torch.cuda.graph(g):
        dattn.dattn_rope(r, x, z, pos)
    del r  # the frequencies went with the capture
    pos.add_(17)
    g.replay()
    torch.cuda.synchronize()
    want2 = torch.empty_like(x)
    dattn.dattn_rope(dattn.Rotation(128), x, want2, pos)
    torch.cuda.synchronize()
    assert torch.equal(z, want2) and not torch.equal(z, want)


# ------------------------------------------------------------------ the rotating append

FORMATS = {"bf16": dattn.KV_BF16, "fp8": dattn.KV_FP8_E4M3, "int4": dattn.KV_INT4,
           "mixed": dattn.KV_MIXED, "block": dattn.KV_FP8_BLOCK}


def _caches(case, fmt, n=2, stats=True):
    kw = dict(head_format=[dattn.KV_FP8_E4M3, dattn.KV_INT4] * (case.Hkv // 2)) \
        if fmt == "mixed" else {}
    out = []
    for _ in range(n):
        c = PagedCache(case, DEV, with_stats=stats, kv_format=FORMATS[fmt], zero_pool=True, **kw)
        out.append(c)
    return out


def _same_state(a, b):
    torch.cuda.synchronize()
    assert int(a.dev_err.item()) == int(b.dev_err.item())
    assert torch.equal(a.seq_lens, b.seq_lens)
    for x, y in ((a.k_pool, b.k_pool), (a.v_pool, b.v_pool), (a.stats, b.stats),
                 (a.kv_scale, b.kv_scale)):
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("d,P,rot,interleaved", [(128, 16, 128, False), (64, 64, 32, True),
                                                 (128, 48, 96, True), (64, 32, 48, False)])
def test_rope_append_is_rope_then_append(fmt, d, P, rot, interleaved):
    r = dattn.Rotation(rot, interleaved=interleaved, scaling="by-parts", factor=4.0)
    case = W.Case("ra", B=3, Hq=12, Hkv=4, d=d, P=P, lens=[0, 131, 47], seed=3,
                  reserve_tokens=400)
    a, b = _caches(case, fmt)
    _same_state(a, b)
    for step, T in enumerate((1, 1, 5, 17, 64, 150)):
        qkv = _rand((case.B, T, 12 + 8, d), 50 + step)
        q, k, v = qkv[:, :, :12], qkv[:, :, 12:16], qkv[:, :, 16:]
        pos = a.seq_lens[:, None] + torch.arange(T, dtype=torch.int32, device=DEV)
        own = step % 2 == 1  # positions given, elsewhere than the slots
        if own:
            pos = pos * 7 + 1000
        want_q, want_k = torch.empty(q.shape, dtype=q.dtype, device=DEV), torch.empty(
            k.shape, dtype=q.dtype, device=DEV)
        dattn.dattn_rope(r, q, want_q, pos.contiguous())
        dattn.dattn_rope(r, k, want_k, pos.contiguous())
        a.append(want_k, v.contiguous())
        got_q = torch.full_like(want_q, float("nan"))
        b.rope_append(r, q, k, v, got_q, positions=pos.contiguous() if own else None)
        _same_state(a, b)
        assert b.seq_lens.tolist() == b.lens
        assert torch.equal(got_q, want_q)


@pytest.mark.parametrize("fmt", ["bf16", "block", "mixed"])
@pytest.mark.parametrize("T", [6, 130])
def test_rope_append_of_a_padded_batch(fmt, T):
    """new_lens: each request's own tokens only; the padding's rows of q_out and of the pool stay."""
    r = dattn.Rotation(64)
    case = W.Case("pad", B=4, Hq=4, Hkv=2, d=64, P=32, lens=[3, 16, 29, 0], seed=4,
                  reserve_tokens=200)
    a, b = _caches(case, fmt)
    counts = [T, 0, T - 1, 3]
    qkv = _rand((4, T, 8, 64), 9)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    got = torch.full(q.shape, 5.0, dtype=q.dtype, device=DEV)
    b.rope_append(r, q, k, v, got, new_lens=counts)
    for i, n in enumerate(counts):
        assert (got[i, n:] == 5.0).all()
        if n == 0:
            continue
        lay = a._row_layout(i)
        qi = torch.empty(1, n, 4, 64, dtype=q.dtype, device=DEV)
        dattn.dattn_rope_append(lay, a.k_pool, a.v_pool, a.stats, r, q[i:i + 1, :n], k[i:i + 1, :n],
                                v[i:i + 1, :n], qi, a.seq_lens[i:i + 1])
        assert torch.equal(qi[0], got[i, :n])
    _same_state(a, b)
    assert b.seq_lens.tolist() == b.lens == [3 + T, 16, 29 + T - 1, 3]
    # a count outside [0, T] is clamped and flagged
    bad = torch.tensor([-1, T + 1, 0, 0], dtype=torch.int32, device=DEV)
    c, = _caches(case, fmt, 1)
    dattn.dattn_rope_append(c.layout, c.k_pool, c.v_pool, c.stats, r, q, k, v, got, c.seq_lens,
                            new_lens=bad, dev_err=c.dev_err)
    torch.cuda.synchronize()
    assert int(c.dev_err.item()) == dattn.DEVERR["LEN_OOB"]
    assert c.seq_lens.tolist() == [3, 16 + T, 29, 0]


@pytest.mark.parametrize("T", [1, 40, 200])
def test_rope_append_without_queries_rotation_or_advance(T):
    case = W.Case("plain", B=2, Hq=4, Hkv=2, d=128, P=16, lens=[20, 7], seed=6, reserve_tokens=256)
    a, b = _caches(case, "bf16")
    k, v = _rand((2, T, 2, 128), 1), _rand((2, T, 2, 128), 2)
    a.append(k, v)
    for _ in range(2):  # without advance a repeated call writes the same slots
        dattn.dattn_rope_append(b.layout, b.k_pool, b.v_pool, b.stats, None, None, k, v, None,
                                b.seq_lens, advance=False, dev_err=b.dev_err)
        assert b.seq_lens.tolist() == case.lens
    b.seq_lens += T
    _same_state(a, b)


def test_rope_append_of_shared_lengths_over_layers():
    """The layers of a model share seq_lens: all but the last leave it, the last advances it."""
    r = dattn.Rotation(128)
    case = W.Case("layers", B=3, Hq=8, Hkv=8, d=128, P=64, lens=[5, 63, 64], seed=7)
    layers = _caches(case, "block", 3, stats=False)
    lens = layers[0].seq_lens
    single = _caches(case, "block", 3, stats=False)
    for step in range(3):
        for i, (c, s) in enumerate(zip(layers, single)):
            q, k, v = (_rand((3, 1, 8, 128), 100 + 10 * step + 3 * i + j) for j in range(3))
            qa, qb = torch.empty_like(q), torch.empty_like(q)
            dattn.dattn_rope_append(c.layout, c.k_pool, c.v_pool, None, r, q, k, v, qa, lens,
                                    advance=i == 2)
            s.rope_append(r, q, k, v, qb)
            assert torch.equal(qa, qb)
    for c, s in zip(layers, single):
        assert torch.equal(c.k_pool, s.k_pool) and torch.equal(c.kv_scale, s.kv_scale)
    assert lens.tolist() == single[0].lens


@pytest.mark.parametrize("fmt", ["bf16", "block"])
def test_rope_append_flags_bad_pages_and_lengths(fmt):
    """Unmapped and foreign pages, a full table and lengths out of range: flagged, nothing else
    written, the other requests served."""
    r = dattn.Rotation(64)
    case = W.Case("bad", B=5, Hq=2, Hkv=2, d=64, P=16, lens=[16] * 5, seed=8, reserve_tokens=16)
    a, b = _caches(case, fmt)
    bt = b.block_table
    bt[0, 1] = -1
    bt[1, 1] = case.num_pages
    b.seq_lens[2] = -5
    b.seq_lens[3] = bt.shape[1] * 16  # no page left
    before = b.k_pool.clone()
    q, k, v = (_rand((5, 1, 2, 64), 20 + i) for i in range(3))
    out = torch.full_like(q, 7.0)
    dattn.dattn_rope_append(b.layout, b.k_pool, b.v_pool, b.stats, r, q, k, v, out, b.seq_lens,
                            dev_err=b.dev_err)
    torch.cuda.synchronize()
    E = dattn.DEVERR
    assert int(b.dev_err.item()) == E["UNMAPPED_PAGE"] | E["PAGE_OOB"] | E["LEN_OOB"]
    assert b.seq_lens.tolist() == [17, 17, -5, bt.shape[1] * 16 + 1, 17]
    assert (out[2] == 7.0).all() and (out[[0, 1, 3, 4]] != 7.0).any(-1).all()
    page = int(bt[4, 1])
    changed = (b.k_pool.view(torch.uint8) != before.view(torch.uint8)).flatten(1).any(1)
    assert changed.nonzero().flatten().tolist() == [page]
    # the same as the good request alone
    dattn.dattn_rope_append(a._row_layout(4), a.k_pool, a.v_pool, a.stats, r, q[4:], k[4:], v[4:],
                            out[4:], a.seq_lens[4:])
    assert torch.equal(a.k_pool[page].view(torch.uint8), b.k_pool[page].view(torch.uint8))


def test_rope_append_in_place_queries_and_nan_keys():
    """q_out may be packed q; a NaN key channel does what dattn_kv_append does with it."""
    r = dattn.Rotation(64)
    case = W.Case("nan", B=2, Hq=4, Hkv=2, d=64, P=16, lens=[0, 9], seed=9)
    a, b = _caches(case, "bf16")
    q, k, v = (_rand((2, 20, h, 64), 30 + h) for h in (4, 2, 2))
    k[:, 0, 0, 3] = float("nan")
    k[:, 9, 1, 40] = float("nan")
    k[:, 12, 1, 5] = float("inf")
    pos = (b.seq_lens[:, None] + torch.arange(20, device=DEV)).to(torch.int32)
    kr, want = torch.empty_like(k), torch.empty_like(q)
    dattn.dattn_rope(r, k, kr, pos)
    dattn.dattn_rope(r, q, want, pos)
    a.append(kr, v)
    b.rope_append(r, q, k, v, q)
    assert torch.equal(q, want)
    _same_state(a, b)


def test_rope_append_captured_and_replayed():
    """One captured step replayed: each replay appends the next token."""
    r = dattn.Rotation(128)
    case = W.Case("graph", B=2, Hq=4, Hkv=2, d=128, P=16, lens=[14, 100], seed=10)
    a, b = _caches(case, "block")
    q, k, v = (_rand((2, 1, h, 128), 40 + h) for h in (4, 2, 2))
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        dattn.dattn_rope_append(b.layout, b.k_pool, b.v_pool, b.stats, r, q, k, v, out, b.seq_lens,
                                dev_err=b.dev_err)
    assert b.seq_lens.tolist() == case.lens
    for i in range(4):
        for j, t in enumerate((q, k, v)):
            t.copy_(_rand(t.shape, 60 + 4 * i + j))
        g.replay()
        want = torch.empty_like(q)
        a.rope_append(r, q, k, v, want)
        assert torch.equal(out, want)
        _same_state(a, b)
