"""The prefill over the block-scaled pool where the lanes of a warp part ways: rows with and without a
query side by side when a cluster's CTAs join their sums, when an accumulator is emptied into the output
rows and when a row is scaled anew. The same call gives the same bits again.

Bound: a weight has a relative error t (its logit: d * 2^-23 of the sum of magnitudes; exponential and
rounding: 2^-20), and between two emptyings 256 products take less than 2^-23 of the sum each, 2^-15
together: t + 2^-15, twice (the sum of the weights and their quotient), of the largest |V|.
"""
import numpy as np
import pytest
import torch

import split_kv_decode_distattention_gb300 as dattn
from split_kv_decode_distattention_gb300 import workloads as W
from split_kv_decode_distattention_gb300.harness import PagedCache

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("Hq,Hkv,d,Tq,lens", [
    (1, 1, 64, 1, [3000, 130, 64, 2048]),     # one row of a tile: half of a joining warp has none
    (2, 1, 64, 67, [5000, 67, 500]),          # a whole query block and three rows
    (4, 1, 128, 5, [20000, 300]),             # emptied in every CTA of a cluster
    (40, 10, 64, 70, [5000, 4097, 71]),       # no clusters: emptied into the output rows
    (24, 24, 128, 129, [2500, 400]),
])
def test_rows_with_and_without_queries_in_a_warp(Hq, Hkv, d, Tq, lens):
    B = len(lens)
    case = W.Case("part", B=B, Hq=Hq, Hkv=Hkv, d=d, P=16, lens=lens, seed=6)
    cache = PagedCache(case, DEV, kv_format=dattn.KV_FP8_BLOCK, zero_pool=True)
    gen = torch.Generator(device=DEV).manual_seed(1)
    # sharp scores for some rows: their maxima climb, so that they are scaled anew while others are not
    q = torch.randn(B, Tq, Hq, d, device=DEV, generator=gen) * torch.tensor([1.0, 5.0, 0.1], device=DEV)[
        torch.arange(Tq, device=DEV) % 3][None, :, None, None]
    q = q.to(torch.bfloat16)
    outs = []
    for _ in range(3):
        out = torch.full((B, Tq, Hq, d), float("nan"), device=DEV)
        m, e = (torch.full((B, Tq, Hq), float("nan"), device=DEV) for _ in range(2))
        dattn.dattn_prefill(cache.layout, cache.k_pool, cache.v_pool, q, case.scale, cache.seq_lens,
                            out, m, e, dev_err=cache.dev_err)
        outs.append((out, m, e))
    torch.cuda.synchronize()
    assert int(cache.dev_err.item()) == 0
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
    out, m, e = outs[0]
    n = case.num_pages * Hkv * (case.P // 16)
    sc = cache.kv_scale[:2 * n].view(case.num_pages, Hkv, case.P // 16, 2).double()
    for b, L in enumerate(lens):
        pages = cache.block_table[b, :-(-L // case.P)].long()
        K, V = ((pool[pages].view(torch.float8_e4m3fn).double() *
                 sc[pages][..., i].repeat_interleave(16, 2)[..., None]).transpose(0, 1).reshape(
                     Hkv, -1, d)[:, :L] for i, pool in enumerate((cache.k_pool, cache.v_pool)))
        see = torch.arange(L, device=DEV)[None] <= (L - Tq + torch.arange(Tq, device=DEV))[:, None]
        for h in range(0, Hq, max(1, Hq // 8)):
            k, v = K[h * Hkv // Hq], V[h * Hkv // Hq]
            x = (q[b, :, h].double() @ k.T * case.scale).masked_fill(~see, -np.inf)
            mag = (q[b, :, h].double().abs() @ k.abs().T * case.scale).masked_fill(~see, 0.0).amax(1)
            t = d * 2.0 ** -23 * mag + 2.0 ** -20
            want = torch.softmax(x, 1) @ v
            most = torch.where(see[..., None], v.abs()[None], 0.0).amax((1, 2))
            err = (out[b, :, h] - want).abs().amax(1)
            assert (err <= 2 * (t + 2.0 ** -15) * most).all(), (b, h)
            assert ((m[b, :, h] - x.amax(1)).abs() <= t + 2.0 ** -22 * x.amax(1).abs()).all()
            lse = torch.logsumexp(x, 1)
            assert ((m[b, :, h] + e[b, :, h].double().log() - lse).abs() <=
                    2 * t + 2.0 ** -22 * lse.abs()).all()
