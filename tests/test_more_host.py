"""The refusals of dattn_decode_shared, dattn_decode_window, dattn_prefill_window and dattn_kv_read, on
the CPU: statuses before any launch, and the binding's checks of its tensors."""
import ctypes

import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import _build

from test_devices_host import on

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FORMATS = (dattn.KV_BF16, dattn.KV_FP8_E4M3, dattn.KV_INT4, dattn.KV_MIXED, dattn.KV_FP8_BLOCK)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return dattn.load_library()


def layout(fmt=dattn.KV_BF16, pages=8, Hkv=2, d=128, P=16, cols=4):
    bt = torch.zeros(1, cols, dtype=torch.int32)
    sc = torch.zeros(4) if fmt != dattn.KV_BF16 else None
    lay = dattn.KVLayout(pages, Hkv, d, P, bt, fmt, sc,
                         [1 + h % 2 for h in range(Hkv)] if fmt == dattn.KV_MIXED else None)
    lay.c.kv_scale = 256 if sc is not None else None
    return lay


P16 = 16  # a pointer that is never followed: the checks fail first


def window(lib, lay=None, q=P16, B=1, T=1, Hq=4, lens=P16, W=5, S=0, splits=0, ws=256, ws_bytes=1 << 30,
           out=P16, bf16=0, k=P16):
    return lib.dattn_decode_window(ctypes.byref((lay or layout()).c), k, P16, q, B, T, Hq, 0.1, lens, W,
                                   S, splits, ws, ws_bytes, out, bf16, None, None, None, None)


def prefill(lib, lay=None, B=1, Tq=1, Hq=4, W=5, S=0, out=P16, bf16=0, q=P16):
    return lib.dattn_prefill_window(ctypes.byref((lay or layout()).c), P16, P16, q, B, Tq, Hq, 0.1, P16,
                                    W, S, out, bf16, None, None, None, None)


def shared(lib, lay=None, B=2, T=1, Hq=4, groups=1, indptr=P16, prefix=P16, ws=256, ws_bytes=1 << 30,
           out=P16, bf16=0, q=P16):
    return lib.dattn_decode_shared(ctypes.byref((lay or layout()).c), P16, P16, q, B, T, Hq, 0.1, P16,
                                   groups, indptr, prefix, ws, ws_bytes, out, bf16, None, None, None,
                                   None)


def read(lib, lay=None, B=1, indptr=P16, lens=P16, N=1, k=P16, ks=256, v=P16, vs=256, f32=0):
    return lib.dattn_kv_read(ctypes.byref((lay or layout()).c), P16, P16, B, indptr, None, lens, N, k, ks,
                             v, vs, f32, None, None)


def test_what_every_call_refuses(lib):
    for call in (window, prefill, shared, read):
        assert call(lib, layout(d=128, P=24)) == UNSUPPORTED
        assert call(lib, layout(pages=1 << 26, P=64)) == UNSUPPORTED
        bad = layout()
        bad.c.head_dim = 96
        assert call(lib, bad) == UNSUPPORTED
        bad = layout()
        bad.c.kv_format = 4
        assert call(lib, bad) == INVALID
        bad = layout(dattn.KV_FP8_BLOCK)
        bad.c.kv_scale = None
        assert call(lib, bad) == INVALID
        bad.c.kv_scale = 8
        assert call(lib, bad) == INVALID
        assert call(lib, B=-1) == INVALID
        assert call(lib, B=5000) == UNSUPPORTED
        assert call(lib, B=0, **({"groups": 0} if call is shared else {})) == OK
    for call in (window, prefill, shared):
        assert call(lib, Hq=3) == INVALID
        assert call(lib, Hq=36) == UNSUPPORTED
        assert call(lib, q=None) == INVALID and call(lib, q=8) == INVALID
        assert call(lib, out=None) == INVALID and call(lib, out=8) == INVALID
        assert call(lib, bf16=2) == INVALID


def test_step_refusals(lib):
    assert window(lib, W=0) == INVALID and window(lib, S=-1) == INVALID
    assert window(lib, T=0) == INVALID and window(lib, splits=-1) == INVALID
    assert window(lib, T=5) == UNSUPPORTED  # g T = 10
    assert window(lib, lens=None) == INVALID and window(lib, k=8) == INVALID
    for fmt in FORMATS:
        # (without a device the workspace is the last check to answer)
        assert window(lib, layout(fmt), T=5) == UNSUPPORTED
    # more tiles than the split counts
    assert window(lib, layout(pages=1 << 10, cols=1 << 22), B=4096, Hq=2, W=1 << 30) == UNSUPPORTED


def test_prefill_refusals(lib):
    assert prefill(lib, W=0) == INVALID and prefill(lib, S=-1) == INVALID
    assert prefill(lib, Tq=-1) == INVALID and prefill(lib, Tq=0) == OK
    assert prefill(lib, Tq=65) == INVALID  # more than the block table holds
    for fmt in (dattn.KV_FP8_E4M3, dattn.KV_INT4, dattn.KV_MIXED):
        assert prefill(lib, layout(fmt)) == UNSUPPORTED


def test_shared_refusals(lib):
    assert shared(lib, T=0) == INVALID and shared(lib, T=5) == UNSUPPORTED
    assert shared(lib, groups=-1) == INVALID
    assert shared(lib, groups=3) == INVALID  # more groups than requests
    assert shared(lib, B=2000, groups=513) == UNSUPPORTED
    assert shared(lib, indptr=None) == INVALID and shared(lib, prefix=None) == INVALID
    for fmt in (dattn.KV_FP8_E4M3, dattn.KV_INT4, dattn.KV_MIXED):
        assert shared(lib, layout(fmt)) == UNSUPPORTED
    n = dattn.dattn_shared_workspace_size(2, 1, 4, 2, 128)
    assert n > 0
    assert shared(lib, ws_bytes=n - 1) == WORKSPACE
    assert shared(lib, ws=None) == WORKSPACE and shared(lib, ws=128) == WORKSPACE
    size = dattn.dattn_shared_workspace_size
    assert size(2, 1, 4, 3, 128) == 0 and size(2, 5, 4, 2, 128) == 0 and size(2, 1, 4, 2, 96) == 0
    assert size(-1, 1, 4, 2, 128) == 0 and size(5000, 1, 4, 2, 128) == 0 and size(2, 0, 4, 2, 128) == 0
    # no group makes it larger, every request and token does
    assert size(3, 1, 4, 2, 128) > n and size(2, 2, 4, 2, 128) > n


def test_read_refusals(lib):
    assert read(lib, N=-1) == INVALID and read(lib, N=0) == OK
    assert read(lib, N=(1 << 30) + 1) == UNSUPPORTED
    assert read(lib, k=None, v=None) == INVALID
    assert read(lib, N=0, k=None, v=None) == OK  # (a tensor without rows has no address)
    assert read(lib, indptr=None) == INVALID and read(lib, lens=None) == INVALID
    assert read(lib, k=8) == INVALID and read(lib, v=8) == INVALID
    assert read(lib, ks=260) == INVALID and read(lib, ks=258, f32=1) == INVALID
    assert read(lib, N=2, vs=248) == INVALID  # rows that overlap
    assert read(lib, f32=2) == INVALID


# ------------------------------------------------------------------------------- the binding

B, T, Hq, Hkv, d, P, PAGES = 2, 3, 4, 2, 64, 16, 8


def tensors():
    z = torch.zeros
    n = PAGES * Hkv * P
    return dict(
        table=z(B, 4, dtype=torch.int32), kv_scale=z(dattn.kv_scale_floats(5, PAGES, Hkv, P)),
        k_pool=z(n * d, dtype=torch.uint8), v_pool=z(n * d, dtype=torch.uint8),
        lens=z(B, dtype=torch.int32), q=z(B, T, Hq, d, dtype=torch.bfloat16), out=z(B, T, Hq, d),
        m=z(B, T, Hq), e=z(B, T, Hq), err=z(1, dtype=torch.int32), ws=z(1 << 12, dtype=torch.uint8),
        ind=z(B + 1, dtype=torch.int32), pre=z(B, dtype=torch.int32), k_out=z(9, Hkv, d),
        v_out=z(9, Hkv, d), starts=z(B, dtype=torch.int32))


class Ws:
    def __init__(self, buffer):
        self.buffer = buffer


def call(name, t):
    lay = dattn.KVLayout(PAGES, Hkv, d, P, t["table"], dattn.KV_FP8_BLOCK, t["kv_scale"])
    pools = lay, t["k_pool"], t["v_pool"]
    if name == "window":
        dattn.dattn_decode_window(*pools, t["q"], 0.1, t["lens"], 5, 1, t["out"], Ws(t["ws"]), t["m"],
                                  t["e"], dev_err=t["err"])
    elif name == "prefill":
        dattn.dattn_prefill_window(*pools, t["q"], 0.1, t["lens"], 5, 1, t["out"], t["m"], t["e"],
                                   dev_err=t["err"])
    elif name == "shared":
        dattn.dattn_decode_shared(*pools, t["q"], 0.1, t["lens"], t["ind"], t["pre"], t["out"],
                                  Ws(t["ws"]), t["m"], t["e"], dev_err=t["err"])
    else:
        dattn.dattn_kv_read(*pools, t["k_out"], t["v_out"], t["ind"], t["lens"], starts=t["starts"],
                            dev_err=t["err"])


POOLS = "k_pool v_pool table kv_scale lens err "
USES = {"window": POOLS + "q out m e ws", "prefill": POOLS + "q out m e",
        "shared": POOLS + "q out m e ws ind pre", "read": POOLS + "ind k_out v_out starts"}


@pytest.fixture
def current(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    # no call may get as far as its launch
    monkeypatch.setattr(dattn, "_check", lambda status, what: pytest.fail(f"{what} was launched"))


@pytest.mark.parametrize("name", USES)
def test_tensors_of_another_device_are_refused(current, name):
    for other in USES[name].split():
        with pytest.raises(ValueError, match="in (one|a) call"):
            call(name, {k: on(v, 1 if k == other else 0) for k, v in tensors().items()})
    with pytest.raises(ValueError, match="in a call on cuda:0"):
        call(name, {k: on(v, 1) for k, v in tensors().items()})
    with pytest.raises(ValueError, match="CUDA"):
        call(name, {k: on(v, -1) for k, v in tensors().items()})


@pytest.mark.parametrize("name", USES)
def test_tensors_too_short_are_refused(current, name):
    # (a shorter out_indptr is a read of fewer requests)
    for other in set(USES[name].split()) - {"err", "ws", "k_out", "v_out", "q"} - \
            ({"ind"} if name == "read" else set()):
        t = tensors()
        t[other] = t[other].reshape(-1)[:-1].reshape(1, -1) if other == "table" else \
            t[other].reshape(-1)[:-1]
        with pytest.raises(ValueError, match="holds"):
            call(name, {k: on(v) for k, v in t.items()})


@pytest.mark.parametrize("name", USES)
def test_types_are_refused(current, name):
    for other in set(USES[name].split()) - {"err", "ws", "table", "kv_scale"}:
        t = tensors()
        t[other] = t[other].to(torch.float64)
        with pytest.raises(TypeError):
            call(name, {k: on(v) for k, v in t.items()})


@pytest.mark.parametrize("name", USES)
def test_tensors_with_gaps_are_refused(current, name):
    for other in set(USES[name].split()) - {"err", "ws", "table", "kv_scale"}:
        t = tensors()
        x = t[other]
        t[other] = torch.zeros(*x.shape, 2, dtype=x.dtype)[..., 0]
        with pytest.raises(ValueError, match="contiguous|packed"):
            call(name, {k: on(v) for k, v in t.items()})


def test_shapes_of_the_read_are_refused(current):
    for bad in (dict(k_out=torch.zeros(9, Hkv, d + 1)), dict(k_out=torch.zeros(9, Hkv + 1, d)),
                dict(v_out=torch.zeros(8, Hkv, d)), dict(k_out=torch.zeros(9, 1, Hkv, d)),
                dict(v_out=torch.zeros(9, Hkv, d, dtype=torch.bfloat16))):
        t = tensors()
        t.update(bad)
        with pytest.raises((ValueError, TypeError)):
            call("read", {k: on(v) for k, v in t.items()})
    t = tensors()
    t["k_out"] = t["v_out"] = None
    with pytest.raises(ValueError):
        call("read", t)
