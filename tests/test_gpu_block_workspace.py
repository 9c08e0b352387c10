"""Workspaces of exactly dattn_workspace_size(..., num_splits) bytes for decodes over the block-scaled
8-bit pool, whose automatic split goes down to four tiles a CTA, and too small ones."""
import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import workloads as W
from split_kv_decode_distattention_gb300.harness import PagedCache

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _decode(cache, q, nbytes, num_splits):
    case = cache.case
    ws = dattn.Workspace(case.B, case.Hq, case.Hkv, case.d, num_splits=num_splits, device=DEV)
    ws.buffer = ws.buffer[:nbytes]
    out = torch.full((case.B, case.Hq, case.d), float("nan"), device=DEV)
    dattn.dattn_decode(cache.layout, cache.k_pool, cache.v_pool, q, case.scale, cache.seq_lens, out,
                       ws, num_splits=num_splits, dev_err=cache.dev_err)
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    return out


@pytest.mark.parametrize("B,Hq,Hkv,d,lens", [(1, 1, 1, 64, [40]), (2, 32, 8, 128, [130, 300]),
                                             (5, 8, 8, 64, [1, 0, 16, 700, 65]),
                                             (3, 16, 2, 128, [20000, 50, 3])])
def test_a_workspace_of_the_stated_size_suffices(B, Hq, Hkv, d, lens):
    case = W.Case("ws", B=B, Hq=Hq, Hkv=Hkv, d=d, P=16, lens=lens, seed=6)
    cache = PagedCache(case, DEV, kv_format=dattn.KV_FP8_BLOCK, zero_pool=True)
    q = torch.randn(B, Hq, d, device=DEV).to(torch.bfloat16)
    size = lambda n: dattn.dattn_workspace_size(B, Hq, Hkv, d, 0, n)  # noqa: E731
    tiles = sum(-(-n // 16) for n in lens) * Hkv
    want = _decode(cache, q, size(1), 1)
    for n in (0, 3, dattn.dattn_auto_splits(tiles)):
        got = _decode(cache, q, size(n), n)
        # the same sums in another order: a relative 2^-20 of values of size 1
        assert (got - want).abs().max().item() <= 2.0 ** -18
    with pytest.raises(dattn.DattnError, match="WORKSPACE"):
        _decode(cache, q, size(3) - 1, 3)
