"""Gathered weights where one block works through many units: runs of units of a single query tile, in which half of the
warps that weigh have nothing to do, before units of several."""
import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from kv8_ref import Paged8, weigh
from streaming_ref import DT, Paged, cu_of, limits

pytestmark = pytest.mark.gpu

# dtype, d, Hq, Hkv, page, causal block, sequences: (how many, new tokens, keys) one after another.  A block takes every
# gridDim-th unit of 256 keys of a head, so each of them meets a run of the short ones before the long ones.
UNITS = [
    ("bf16", 128, 8, 8, 64, 0, [(48, 40, 300), (12, 500, 512), (30, 70, 130), (10, 257, 400)]),
    ("fp16", 64, 16, 4, 16, 1, [(60, 30, 511), (10, 130, 300), (70, 9, 90), (16, 100, 480)]),
    ("bf16", 64, 12, 12, 129, 0, [(90, 128, 128), (9, 384, 700), (20, 128, 257), (7, 1000, 1001)]),
    ("fp16", 128, 6, 2, 200, 16, [(200, 42, 100), (40, 43, 260), (8, 600, 600)]),
]


@pytest.mark.parametrize("case", UNITS, ids=lambda c: f"{c[0]}-d{c[1]}-{c[2]}over{c[3]}-page{c[4]}-block{c[5]}")
@pytest.mark.parametrize("bits", [16, 8])
def test_runs_of_units_of_one_query_tile(case, bits):
    dtype, d, Hq, Hkv, page, block, runs = case
    dt = DT[dtype]
    # lengths within a run differ by a few, so that its units are not all alike
    news = [max(1, n - i % 3) for count, n, _ in runs for i in range(count)]
    lens = [max(new, L - i % 5) for (new, L, i) in zip(news, [L for c, _, L in runs for _ in range(c)], range(len(news)))]
    if bits == 8:
        c = Paged8(d, Hkv, page, lens, 201)
        cache, keys = c.cache(vdx), lambda s: c.get(c.k, c.k_scale, s)
    else:
        c = Paged(dt, d, Hkv, page, lens, 201)
        cache, keys = vdx.PagedKV(c.k, c.v, c.table), lambda s: c.get(s)[0].double()
    g = torch.Generator(device="cuda").manual_seed(202)
    q = (torch.randn(sum(news), Hq, d, generator=g, device="cuda") * 0.7).to(dt)
    cu = cu_of(news)
    bounds = dict(max_q=max(news), max_kv=max(lens), causal_block=block)
    _, lse = vdx.paged_attn(q, cache, cu, c.kv_len, **bounds)
    w = torch.rand(len(lens), Hkv, max(lens) + 3, generator=g, device="cuda")
    before, again = w.clone(), [w.clone() for _ in range(5)]
    vdx.paged_attn_weights(q, cache, cu, c.kv_len, lse, w, decay=0.5, **bounds)
    for x in again:
        vdx.paged_attn_weights(q, cache, cu, c.kv_len, lse, x, decay=0.5, **bounds)
    vdx.sync_check()
    assert all(torch.equal(x, w) for x in again)
    at = 0
    for s, (n, L) in enumerate(zip(news, lens)):
        want = before[s, :, :L].double() * 0.5
        want[:, L - n:] = 0
        bound = 2.0 ** -22 * want
        add, b = weigh(q[at:at + n], keys(s), limits(n, L, block), lse[:, at:at + n])
        want += add
        bound += b + 2.0 ** -22 * want
        err = (w[s, :, :L].double() - want).abs()
        assert bool((err <= bound).all()), (s, float((err / bound).max()))
        at += n
    past = torch.arange(w.shape[2], device="cuda")[None, None] >= c.kv_len[:, None, None]
    assert torch.equal(w[past.expand_as(w)], before[past.expand_as(w)])
