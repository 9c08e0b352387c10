"""Every call refuses tensors of another device than the current one before anything is launched. On the
CPU: tensors that only say which GPU they are on."""
import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import _build


class On(torch.Tensor):
    """A CPU tensor that answers get_device() with `gpu`."""

    gpu = 0

    def get_device(self):
        return self.gpu


def on(t, gpu=0):
    t = torch.Tensor._make_subclass(On, t)
    t.gpu = gpu
    return t


@pytest.fixture(autouse=True)
def current(monkeypatch):
    _build.build()
    dattn.load_library()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    # no call may get as far as its launch
    monkeypatch.setattr(dattn, "_check", lambda status, what: pytest.fail(f"{what} was launched"))


B, T, Hq, Hkv, d, P, PAGES = 2, 3, 4, 2, 64, 16, 8


def _tensors():
    z = torch.zeros
    n = PAGES * Hkv * P
    return dict(
        table=z(B, 4, dtype=torch.int32), kv_scale=z(dattn.kv_scale_floats(5, PAGES, Hkv, P)),
        k_pool=z(n * d, dtype=torch.uint8), v_pool=z(n * d, dtype=torch.uint8),
        stats=z(n // 16 * 2 * d, dtype=torch.bfloat16), lens=z(B, dtype=torch.int32),
        new=z(B, 1, Hkv, d, dtype=torch.bfloat16), q=z(B, Hq, d, dtype=torch.bfloat16),
        qt=z(B, T, Hq, d, dtype=torch.bfloat16), out=z(B, T, Hq, d), m=z(B, T, Hq), e=z(B, T, Hq),
        err=z(1, dtype=torch.int32), ws=z(1 << 12, dtype=torch.uint8),
        kind=z(Hkv, dtype=torch.int8), sel=z(B, Hkv, 2, dtype=torch.int32),
        lists=z(B, Hkv, 3, 2, dtype=torch.int32), req=z(2, dtype=torch.int32),
        ind=z(3, dtype=torch.int32), pages=z(2, dtype=torch.int32), MA=z(2, Hq, d),
        MAr=z(2, B, Hq, d))


class _Workspace:
    def __init__(self, buffer):
        self.buffer = buffer


def _call(name, t):
    fmt = dattn.KV_FP8_BLOCK
    lay = dattn.KVLayout(PAGES, Hkv, d, P, t["table"], fmt, t["kv_scale"])
    ws = _Workspace(t["ws"])
    sp = dattn.SparseConfig(t["kind"], 4, 8, 2, t["sel"])
    pools = lay, t["k_pool"], t["v_pool"]
    tail = dict(dev_err=t["err"])
    if name == "kv_append":
        dattn.dattn_kv_append(*pools, t["stats"], t["new"], t["new"], t["lens"], **tail)
    elif name == "decode":
        dattn.dattn_decode(*pools, t["q"], 0.1, t["lens"], t["out"], ws, t["m"], t["e"], sp, **tail)
    elif name == "decode_noalloc":
        dattn.dattn_decode_noalloc(*pools, t["q"], 0.1, t["lens"], t["out"], t["m"], t["e"], sp, **tail)
    elif name == "append_decode":
        dattn.dattn_append_decode(*pools, t["stats"], t["new"], t["new"], t["q"], 0.1, t["lens"],
                                  t["out"], ws, t["m"], t["e"], sp, **tail)
    elif name == "decode_multi":
        dattn.dattn_decode_multi(*pools, t["qt"], 0.1, t["lens"], t["out"], ws, t["m"], t["e"], **tail)
    elif name == "prefill":
        pf = dattn.PrefillSparseConfig(t["kind"], 1, 1, t["lists"])
        dattn.dattn_prefill(*pools, t["qt"], 0.1, t["lens"], t["out"], t["m"], t["e"], pf, **tail)
    elif name == "partial":
        dattn.dattn_partial(*pools, t["q"], 0.1, t["lens"], t["req"], t["ind"], t["pages"], t["m"],
                            t["e"], t["MA"], ws, **tail)
    elif name == "merge":
        dattn.dattn_merge(t["ind"], t["m"], t["e"], t["MA"], t["out"], **tail)
    elif name == "merge_gathered":
        dattn.dattn_merge_gathered(t["m"], t["e"], t["MAr"], t["out"], **tail)
    elif name == "page_select":
        dattn.dattn_page_select(lay, t["stats"], t["q"], t["lens"], t["kind"], 2, t["sel"], ws, **tail)


POOLS = "k_pool v_pool table kv_scale lens err "
USES = {
    "kv_append": POOLS + "stats new", "decode": POOLS + "q out m e ws kind sel",
    "decode_noalloc": POOLS + "q out m e kind sel",
    "append_decode": POOLS + "stats new q out m e ws kind sel",
    "decode_multi": POOLS + "qt out m e ws", "prefill": POOLS + "qt out m e kind lists",
    "partial": POOLS + "q req ind pages m e MA ws", "merge": "ind m e MA out err",
    "merge_gathered": "m e MAr out err", "page_select": "stats q lens kind sel ws table err",
}


@pytest.mark.parametrize("name", USES)
def test_a_call_with_a_tensor_of_another_device_is_refused(name):
    for other in USES[name].split():
        t = {k: on(v, 1 if k == other else 0) for k, v in _tensors().items()}
        with pytest.raises(ValueError, match="in (one|a) call"):
            _call(name, t)


@pytest.mark.parametrize("name", USES)
def test_a_call_on_another_device_than_the_current_one_is_refused(name):
    with pytest.raises(ValueError, match="in a call on cuda:0"):
        _call(name, {k: on(v, 1) for k, v in _tensors().items()})


@pytest.mark.parametrize("name", USES)
def test_a_call_with_tensors_of_the_host_is_refused(name):
    with pytest.raises(ValueError, match="CUDA"):
        _call(name, {k: on(v, -1) for k, v in _tensors().items()})
