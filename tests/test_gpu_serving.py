"""The calls together, as a server makes them: a prompt through a window, its pages shared by the requests
that follow, decode steps behind the shared prefix and through a window, and the cache read back."""
import numpy as np
import pytest
import torch

from _block_ref import attention
from _paged import check, weight_error

pytestmark = pytest.mark.gpu

DEV = "cuda"
B, Hq, Hkv, d, P, PREFIX, W, S = 5, 8, 2, 128, 16, 208, 64, 4


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("name", ("bf16", "fp8-block"))
def test_prompt_shared_by_requests_decoded_and_read_back(name):
    import split_kv_decode_distattention_gb300 as dattn
    fmt = dattn.KV_BF16 if name == "bf16" else dattn.KV_FP8_BLOCK
    pages, cols, scale = 64, PREFIX // P + 4, d ** -0.5
    g = torch.Generator(device=DEV).manual_seed(7)

    def rnd(*shape):
        return torch.randn(*shape, d, device=DEV, generator=g).to(torch.bfloat16)

    kp, vp = (torch.zeros(pages * Hkv * P * d, device=DEV,
                          dtype=torch.bfloat16 if name == "bf16" else torch.uint8) for _ in range(2))
    sc = torch.zeros(max(dattn.kv_scale_floats(fmt, pages, Hkv, P), 4), device=DEV)
    err = i32([0])
    rot = dattn.Rotation(d)

    def layout(table):
        return dattn.KVLayout(pages, Hkv, d, P, i32(table), fmt, sc)

    def values(lay, lens):
        """K and V of every request as the cache holds them, read back in fp32."""
        ends = np.concatenate([[0], np.cumsum(lens)])
        k, v = (torch.empty(int(ends[-1]), Hkv, d, device=DEV) for _ in range(2))
        dattn.dattn_kv_read(lay, kp, vp, k, v, i32(ends.tolist()), i32(lens), dev_err=err)
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        return [(k[a:b], v[a:b]) for a, b in zip(ends[:-1], ends[1:])]

    def compare(out, q, kv, lens, see, what):
        for b, (K, V) in enumerate(kv):
            for h in range(Hq):
                ref, _, _, bound, _ = attention(q[b, :, h].double().cpu().numpy(), K[:, h // 4],
                                                V[:, h // 4], scale, see(lens[b]), weight_error("bf16"))
                check(out[b, :, h], None, None, ref, bound, 0, 0, 0, f"{what} b={b} h={h}")

    # the prompt: appended with its rotation, attended through the window
    prompt = layout([list(range(PREFIX // P)) + [-1] * 4])
    lens = i32([0])
    q = torch.empty(1, PREFIX, Hq, d, dtype=torch.bfloat16, device=DEV)
    dattn.dattn_rope_append(prompt, kp, vp, None, rot, rnd(1, PREFIX, Hq), rnd(1, PREFIX, Hkv),
                            rnd(1, PREFIX, Hkv), q, lens, dev_err=err)
    out = torch.empty(1, PREFIX, Hq, d, device=DEV)
    dattn.dattn_prefill_window(prompt, kp, vp, q, scale, lens, W, S, out, dev_err=err)

    def window(T):
        def see(L):
            p, i = np.arange(L - T, L)[:, None], np.arange(L)[None]
            return (i <= p) & ((i > p - W) | (i < S))
        return see

    compare(out, q, values(prompt, [PREFIX]), [PREFIX], window(PREFIX), "prompt")
    # five requests behind it, each with pages of its own; three steps of two tokens
    table = [list(range(PREFIX // P)) + [PREFIX // P + 4 * b + j for j in range(4)] for b in range(B)]
    lay, lens = layout(table), i32([PREFIX] * B)
    ws, ws2 = dattn.SharedWorkspace(B, 2, Hq, Hkv, d), dattn.Workspace(B, 2 * Hq, Hkv, d)
    for step in range(3):
        q = torch.empty(B, 2, Hq, d, dtype=torch.bfloat16, device=DEV)
        dattn.dattn_rope_append(lay, kp, vp, None, rot, rnd(B, 2, Hq), rnd(B, 2, Hkv), rnd(B, 2, Hkv), q,
                                lens, dev_err=err)
        now = [PREFIX + 2 * (step + 1)] * B
        assert lens.tolist() == now
        shared, near, full = (torch.empty(B, 2, Hq, d, device=DEV) for _ in range(3))
        dattn.dattn_decode_shared(lay, kp, vp, q, scale, lens, i32([0, B]), i32([PREFIX]), shared, ws,
                                  dev_err=err)
        dattn.dattn_decode_window(lay, kp, vp, q, scale, lens, W, S, near, ws2, dev_err=err)
        dattn.dattn_decode_multi(lay, kp, vp, q, scale, lens, full, ws2, dev_err=err)
        kv = values(lay, now)
        causal = lambda L: np.arange(L)[None] <= np.arange(L - 2, L)[:, None]  # noqa: E731
        compare(shared, q, kv, now, causal, "shared")
        compare(full, q, kv, now, causal, "full")
        compare(near, q, kv, now, window(2), "window")
    assert int(err) == 0


def test_on_another_stream_than_the_current_one():
    """Every call on a stream of its own, behind work that the stream has to wait for."""
    import split_kv_decode_distattention_gb300 as dattn
    from _paged import Paged
    pool = Paged("bf16", [300, 290, 280], 2, 64, 16, seed=5, shared=[(0, 3, 256)])
    lay, (kp, vp) = pool.layout(dattn), pool.pools()
    g = torch.Generator(device=DEV).manual_seed(1)
    src = torch.randn(3, 2, 4, 64, device=DEV, generator=g).to(torch.bfloat16)
    lens, ends, told = i32(pool.lens), i32([0, 3]), i32([256])
    ws, ws2 = dattn.SharedWorkspace(3, 2, 4, 2, 64), dattn.Workspace(3, 8, 2, 64)
    k = torch.empty(870, 2, 64, device=DEV)
    at = i32([0, 300, 590, 870])

    def run(q, outs, k, stream):
        a, b, c = outs
        dattn.dattn_decode_shared(lay, kp, vp, q, 0.1, lens, ends, told, a, ws, stream=stream)
        dattn.dattn_decode_window(lay, kp, vp, q, 0.1, lens, 33, 2, b, ws2, stream=stream)
        dattn.dattn_prefill_window(lay, kp, vp, q, 0.1, lens, 33, 2, c, stream=stream)
        dattn.dattn_kv_read(lay, kp, vp, k, None, at, lens, stream=stream)

    want = [torch.empty(3, 2, 4, 64, device=DEV) for _ in range(3)]
    run(src, want, k, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, k2 = torch.zeros_like(src), torch.empty_like(k)
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        q.copy_(src)
    run(q, outs, k2, s)
    s.synchronize()
    for x, y in zip(outs + [k2], want + [k]):
        assert torch.equal(x, y)
