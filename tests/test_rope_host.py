"""The rotation's host side and the refusals of the rotary and block-scaled calls, on the CPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import _build

import _block_ref as ref

INVALID, UNSUPPORTED = 1, 2
PTR = ctypes.c_void_p(4096)  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return dattn.load_library()


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
def test_frequencies_of_each_scaling(rot):
    n, base = rot // 2, 500000.0
    f = base ** (-2.0 * np.arange(n) / rot)
    # pow is within an ulp of its value on both machines: a few ulps
    tol = dict(rtol=2.0 ** -48, atol=0)
    np.testing.assert_allclose(dattn.dattn_rope_frequencies(rot, base), f, **tol)
    np.testing.assert_allclose(dattn.dattn_rope_frequencies(rot, base, "linear", 8.0), f / 8, **tol)
    b2 = base * 8.0 ** (rot / (rot - 2))
    np.testing.assert_allclose(dattn.dattn_rope_frequencies(rot, base, "ntk", 8.0),
                               b2 ** (-2.0 * np.arange(n) / rot), **tol)
    got = dattn.dattn_rope_frequencies(rot, base, "by-parts", 8.0, original_len=8192, low=1, high=4)
    turns = 8192 * f / (2 * math.pi)
    for g, t, x in zip(got, turns, f):
        w = min(1.0, max(0.0, (t - 1) / 3))
        assert g == pytest.approx(x * (w + (1 - w) / 8), rel=2.0 ** -45)
        if t >= 4:
            assert g == pytest.approx(x, rel=2.0 ** -48)
        if t <= 1:
            assert g == pytest.approx(x / 8, rel=2.0 ** -48)


def test_turns_are_the_fraction_of_a_turn():
    f = [1.0, 0.1, 1e-5, 2 * math.pi, 7.0, -0.25, 0.0]
    r = dattn.Rotation(16, inv_freq=f + [3.0])
    for t, x in zip(list(r._turns), f):
        want = float((ref.Fraction(x) / ref.TWO_PI) % 1)
        d = abs(t / 2.0 ** 64 - want)
        assert min(d, 1 - d) <= 2.0 ** -51  # the double quotient's rounding, |x| < 8


def test_rotation_refuses_bad_arguments():
    for kw in (dict(base=0.0), dict(base=float("nan")), dict(scaling="linear", factor=0.0),
               dict(scaling="by-parts", factor=2.0, low=4.0, high=4.0),
               dict(scaling="by-parts", factor=2.0, original_len=0.0)):
        with pytest.raises(dattn.DattnError):
            dattn.Rotation(32, **kw)
    with pytest.raises(ValueError):
        dattn.Rotation(32, scaling="dynamic")
    with pytest.raises(ValueError):
        dattn.Rotation(32, inv_freq=[1.0] * 15)
    with pytest.raises(dattn.DattnError):
        dattn.Rotation(32, inv_freq=[float("inf")] * 16)
    with pytest.raises(dattn.DattnError):
        dattn.Rotation(24)  # not a multiple of 16


def _rope(lib, rot, x=PTR, xs=512, out=PTR, os_=512, N=4, H=4, d=128, f32=0, pos=PTR, inv=0):
    return lib.dattn_rope(ctypes.byref(rot) if rot is not None else None, x, xs, out, os_, N, H, d,
                          f32, pos, inv, None)


def test_rope_refuses_bad_calls(lib):
    r = dattn.Rotation(64).c

    def rot(**kw):
        c = dattn._Rotation(64, 0, 1.0, r.turns)
        for k, v in kw.items():
            setattr(c, k, v)
        return c

    assert _rope(lib, None) == INVALID
    assert _rope(lib, rot(rot_dim=-16)) == INVALID
    assert _rope(lib, rot(rot_dim=144)) == INVALID
    assert _rope(lib, rot(rot_dim=128), d=64, xs=256, os_=256) == INVALID
    assert _rope(lib, rot(rot_dim=40)) == UNSUPPORTED
    assert _rope(lib, rot(interleaved=2)) == INVALID
    assert _rope(lib, rot(amplitude=float("nan"))) == INVALID
    assert _rope(lib, rot(turns=None)) == INVALID
    assert _rope(lib, r, d=96) == UNSUPPORTED
    assert _rope(lib, r, d=0) == INVALID
    assert _rope(lib, r, H=0) == INVALID
    assert _rope(lib, r, H=5000) == UNSUPPORTED
    assert _rope(lib, r, N=-1) == INVALID
    assert _rope(lib, r, N=0, x=None) == 0  # nothing to do
    assert _rope(lib, r, x=None) == INVALID
    assert _rope(lib, r, pos=None) == INVALID
    assert _rope(lib, r, x=ctypes.c_void_p(4104)) == INVALID  # misaligned
    assert _rope(lib, r, xs=516) == INVALID
    assert _rope(lib, r, xs=504) == INVALID  # tokens would overlap
    assert _rope(lib, r, os_=1024) == INVALID  # in place with two strides
    assert _rope(lib, r, f32=2) == INVALID
    assert _rope(lib, r, inv=-1) == INVALID


def _layout(fmt=0, scale=None, **kw):
    bt = torch.zeros(1, 4, dtype=torch.int32)
    a = dict(num_pages=8, num_kv_heads=2, head_dim=128, page_size=16)
    a.update(kw)
    lay = dattn.KVLayout(a["num_pages"], a["num_kv_heads"], a["head_dim"], a["page_size"], bt)
    lay.c.kv_format, lay.c.kv_scale = fmt, scale
    return lay


def _append(lib, lay, rot=None, q=PTR, qs=512, k=PTR, ks=256, v=PTR, vs=256, B=2, T=3, Hq=4,
            q_out=ctypes.c_void_p(8192), lens=PTR, advance=1, pool=PTR):
    return lib.dattn_rope_append(ctypes.byref(lay.c), pool, pool, None, rot, q, qs, k, ks, v, vs, B,
                                 T, Hq, q_out, lens, None, None, advance, None, None)


def test_rope_append_refuses_bad_calls(lib):
    lay = _layout()
    r = dattn.Rotation(64)
    assert _append(lib, lay, B=-1) == INVALID
    assert _append(lib, lay, T=-1) == INVALID
    assert _append(lib, lay, T=0) == 0
    assert _append(lib, lay, B=0) == 0
    assert _append(lib, lay, Hq=0) == INVALID  # queries without heads
    assert _append(lib, lay, Hq=5000, qs=1 << 20) == UNSUPPORTED
    assert _append(lib, lay, q=None) == INVALID  # q_out without q
    assert _append(lib, lay, q_out=None) == INVALID
    assert _append(lib, lay, k=None) == INVALID
    assert _append(lib, lay, lens=None) == INVALID
    assert _append(lib, lay, pool=None) == INVALID
    assert _append(lib, lay, ks=248) == INVALID
    assert _append(lib, lay, vs=260) == INVALID
    assert _append(lib, lay, qs=504) == INVALID
    assert _append(lib, lay, qs=1024, q_out=PTR) == INVALID  # in place, not packed
    assert _append(lib, lay, advance=3) == INVALID
    assert _append(lib, lay, v=ctypes.c_void_p(4098)) == INVALID
    assert _append(lib, lay, B=70000) == UNSUPPORTED
    bad = dattn._Rotation(144, 0, 1.0, r.c.turns)
    assert _append(lib, lay, rot=ctypes.byref(bad)) == INVALID
    assert _append(lib, _layout(head_dim=96)) == UNSUPPORTED


def test_block_scaled_layout_is_validated(lib):
    F = dattn.KV_FP8_BLOCK
    dec = lambda lay, Hq=4: lib.dattn_decode(  # noqa: E731
        ctypes.byref(lay.c), PTR, PTR, PTR, 1, Hq, 0.1, PTR, None, 0, PTR, 1 << 20, PTR, None,
        None, None, None)
    assert dec(_layout(F, None)) == INVALID  # no scales
    assert dec(_layout(F, 72)) == INVALID  # misaligned scales
    assert dec(_layout(F, 128), Hq=36) == UNSUPPORTED  # passes the layout checks
    # the fused append and decode does not take the format
    assert lib.dattn_append_decode(ctypes.byref(_layout(F, 128).c), PTR, PTR, None, PTR, PTR, PTR,
                                   1, 4, 0.1, PTR, None, 0, PTR, 1 << 20, PTR, None, None, None,
                                   None) == UNSUPPORTED
    with pytest.raises(ValueError):
        dattn.KVLayout(8, 2, 128, 16, torch.zeros(1, 4, dtype=torch.int32), kv_format=F)


def test_scale_floats_are_padded():
    F = dattn.KV_FP8_BLOCK
    assert dattn.kv_scale_floats(F, 1, 1, 16) == 4
    assert dattn.kv_scale_floats(F, 3, 1, 16) == 8
    assert dattn.kv_scale_floats(F, 4, 2, 64) == 64
    assert dattn.kv_scale_floats(dattn.KV_FP8_E4M3, 4, 2, 64) == 1024
    assert dattn.kv_scale_floats(dattn.KV_BF16, 4, 2, 64) == 0


def test_the_binding_refuses_tensors_that_do_not_fit():
    r = dattn.Rotation(64)
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        dattn.dattn_rope(r, x.half(), x.half(), pos)
    with pytest.raises(TypeError):
        dattn.dattn_rope(r, x, x.float(), pos)
    with pytest.raises(TypeError):
        dattn.dattn_rope(r, x, x, pos.long())
    with pytest.raises(ValueError):
        dattn.dattn_rope(r, x, x[:1], pos)
    with pytest.raises(ValueError):
        dattn.dattn_rope(r, x, x, pos[:1])
    # tokens that are not evenly spaced, heads that are not packed
    y = torch.zeros(2, 6, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="evenly spaced"):
        dattn._tokens(y[:, :4], "x")
    with pytest.raises(ValueError, match="packed"):
        dattn._tokens(y[:, :, ::2], "x")
    with pytest.raises(ValueError, match="CUDA"):
        dattn._tokens(y, "x")


def test_reference_block_scale_is_the_formulas():
    """The reference's scale against the inequality it comes from."""
    rng = np.random.default_rng(5)
    for m in np.exp2(rng.uniform(-100, 100, 200)):
        s = ref.block_scale(m)
        assert m <= 448 * s and m > 224 * s and math.log2(s) == int(math.log2(s))
    assert ref.block_scale(448.0) == 1.0 and ref.block_scale(450.0) == 2.0
    assert ref.block_scale(0.0) == 0.0
    assert ref.block_scale(1e-45) == 2.0 ** -126
    assert ref.block_scale(math.inf) == 2.0 ** 119
