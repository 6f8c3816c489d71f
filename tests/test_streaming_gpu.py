"""Paged-cache append, paged attention and cross attention on the GPU (through the public calls)
against plain 64-bit forms, with bounds derived from the arithmetic (tests/streaming_ref.py)."""
import math

import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from streaming_ref import (DT, SECTIONS, Paged, attend, check_attention, cu_of, limits, rotate, rotate_bound)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from video_diffusion_transformer_rope_gb300 import _build
    _build.build()
    vdx.lib()


def _rand(shape, dtype, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


# ------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,d,Hq,Hkv,page,news,ctxs,grid,norm,order", [
    ("bf16", 128, 12, 12, 16, [1, 1, 1], [0, 15, 500], (2000, 1, 1), True, "token"),
    ("bf16", 128, 3, 3, 130, [131, 0, 77], [0, 5, 129], (40, 5, 7), True, "head"),
    ("fp16", 64, 12, 4, 32, [5, 33, 1, 64, 2], [31, 0, 32, 7, 1000], (2000, 1, 1), False, "token"),
    ("fp16", 128, 5, 1, 64, [70], [0], (9, 3, 3), True, "token"),
    ("bf16", 64, 40, 8, 200, [3, 400], [199, 1], (900, 1, 2), False, "head"),
    ("bf16", 128, 2, 2, 1560, [1560, 10], [1560, 3119], (21, 30, 52), True, "token"),
])
def test_append_matches_the_formula(dtype, d, Hq, Hkv, page, news, ctxs, grid, norm, order):
    dt = DT[dtype]
    lens = [a + b for a, b in zip(news, ctxs)]
    c = Paged(dt, d, Hkv, page, lens, seed=1, order=order)
    kc0, vc0 = c.k.clone(), c.v.clone()
    n = sum(news)
    qkv = _rand((n + 2, Hq + 2 * Hkv, d), dt, 2, 2.0)           # two rows behind the last sequence
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    wq, wk = (_rand((d,), dt, 3) if norm else None), (_rand((d,), dt, 4) if norm else None)
    q_out = torch.full((n + 2, Hq, d), 9.0, dtype=dt, device="cuda")
    r = vdx.rope3d_append(q, k, v, vdx.PagedKV(c.k, c.v, c.table), cu_of(news), c.kv_len, grid, SECTIONS[d], q_norm=wq,
                          k_norm=wk, eps=1e-5, q_out=q_out)
    vdx.sync_check()
    assert r is q_out and bool((q_out[n:] == 9.0).all())
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    at = 0
    for s, (m, before) in enumerate(zip(news, ctxs)):
        rows = slice(at, at + m)
        pos = torch.arange(before, before + m, device="cuda")
        for got, x, w in ((q_out[rows], q[rows], wq), (c.k[c.slots(s, pos)], k[rows], wk)):
            ref = rotate(x, pos, grid, SECTIONS[d], 10000.0, w, 1e-5)
            err = (got.double() - ref).abs()
            assert bool((err <= rotate_bound(ref, dt)).all()), float((err / rotate_bound(ref, dt)).max())
        assert torch.equal(c.v[c.slots(s, pos)], v[rows])
        touched[c.slots(s, pos)] = True
        at += m
    for now, was in ((c.k, kc0), (c.v, vc0)):                    # every other slot is as it was
        assert torch.equal(now[~touched].view(torch.int16), was[~touched].view(torch.int16))


def test_append_far_positions_keep_their_angles():
    # position 5e8 of a one-axis grid: an fp32 product would lose the angle altogether
    c = Paged(torch.float16, 128, 1, 16, [1, 1], seed=5)
    off = torch.tensor([500_000_003, 77_777], dtype=torch.int32, device="cuda")
    q, k, v = (_rand((2, 1, 128), torch.float16, s) for s in (6, 7, 8))
    grid = (2_000_000_000, 1, 1)
    got = vdx.rope3d_append(q, k, v, vdx.PagedKV(c.k, c.v, c.table), cu_of([1, 1]), c.kv_len, grid, (128, 0, 0), pos_offset=off)
    vdx.sync_check()
    ref = rotate(q, off.long(), grid, (128, 0, 0), 10000.0)
    # the 64-bit product of the plain form is itself off by half a unit of its 53 bits: 5e8 * 2^-53
    assert bool(((got.double() - ref).abs() <= rotate_bound(ref, torch.float16) + 6e-8 * ref.abs().amax()).all())


def test_append_in_place_and_without_queries():
    news, lens = [3, 9], [20, 9]
    a, b = (Paged(torch.bfloat16, 128, 2, 16, lens, seed=9) for _ in range(2))
    qkv = _rand((12, 2 + 4, 128), torch.bfloat16, 10)
    q, k, v = qkv[:, :2], qkv[:, 2:4], qkv[:, 4:]
    grid = (30, 1, 1)
    want = vdx.rope3d_append(q, k, v, vdx.PagedKV(a.k, a.v, a.table), cu_of(news), a.kv_len, grid)
    assert vdx.rope3d_append(None, k, v, vdx.PagedKV(b.k, b.v, b.table), cu_of(news), b.kv_len, grid) is None
    assert torch.equal(a.k.nan_to_num(), b.k.nan_to_num()) and torch.equal(a.v.nan_to_num(), b.v.nan_to_num())
    before = qkv[:, 2:].clone()
    vdx.rope3d_append(q, k, v, vdx.PagedKV(b.k, b.v, b.table), cu_of(news), b.kv_len, grid, q_out=q)
    vdx.sync_check()
    assert torch.equal(q, want) and torch.equal(qkv[:, 2:], before)


@pytest.mark.parametrize("layout", ["kinds", "kinds_of_a_head", "padded"])
def test_append_in_place_within_a_fused_projection(layout):
    dt, d, H, n, grid = torch.bfloat16, 128, 3, 40, (40, 1, 1)
    if layout == "kinds":                                            # [rows, 3, H, d]
        x = _rand((n, 3, H, d), dt, 60)
        q, k, v = x.unbind(1)
    elif layout == "kinds_of_a_head":                                # [rows, H, 3, d]
        x = _rand((n, H, 3, d), dt, 61)
        q, k, v = x.unbind(2)
    else:                                                            # v, q, k and a gap
        x = _rand((n, 3 * H + 1, d), dt, 62)
        v, q, k = x[:, :H], x[:, H:2 * H], x[:, 2 * H:3 * H]
    before = [t.clone() for t in (q, k, v)]
    c = Paged(dt, d, H, 16, [n], seed=63)
    r = vdx.rope3d_append(q, k, v, vdx.PagedKV(c.k, c.v, c.table), cu_of([n]), c.kv_len, grid, SECTIONS[d], q_out=q)
    vdx.sync_check()
    pos = torch.arange(n, device="cuda")
    ref = rotate(before[0], pos, grid, SECTIONS[d], 10000.0, None, 1e-6)
    assert r is q and bool(((q.double() - ref).abs() <= rotate_bound(ref, dt)).all())
    assert torch.equal(k, before[1]) and torch.equal(v, before[2]) and torch.equal(c.v[c.slots(0, pos)], v)


def test_append_of_queries_without_heads_is_refused():
    c = Paged(torch.bfloat16, 128, 2, 16, [5], seed=64)
    x = _rand((5, 2, 128), torch.bfloat16, 65)
    with pytest.raises(vdx.VdxError):
        vdx.rope3d_append(x[:, :0], x, x, vdx.PagedKV(c.k, c.v, c.table), cu_of([5]), c.kv_len, (5, 1, 1))


def test_sizes_past_32_bits_are_refused():
    # broadcast views: nothing of this size is in memory
    n, dt = 2 ** 32 + 1, torch.bfloat16
    x = torch.zeros(1, 1, 1, 128, dtype=dt, device="cuda")
    long = x.expand(1, n, 1, 128)
    out = torch.empty(1, 1, 1, 128, dtype=dt, device="cuda")
    with pytest.raises(vdx.VdxError):
        vdx.cross_attn(x, long, long, out=out)
    pages = torch.zeros(1, 16, 1, 128, dtype=dt, device="cuda")
    cu, one = cu_of([1]), torch.ones(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for cache in (vdx.PagedKV(pages.expand(n, -1, -1, -1), pages.expand(n, -1, -1, -1), table),
                  vdx.PagedKV(pages, pages.clone(), table.expand(n, 1))):
        with pytest.raises(vdx.VdxError):
            vdx.paged_attn(x[0], cache, cu, one)


def test_append_skips_and_reports_what_has_no_place():
    c = Paged(torch.bfloat16, 64, 1, 16, [20, 4], seed=11)
    k0 = c.k.clone()
    k = _rand((6, 1, 64), torch.bfloat16, 12)
    q = _rand((6, 1, 64), torch.bfloat16, 13)
    cache = vdx.PagedKV(c.k, c.v, c.table)
    good = c.table.clone()
    c.table[0, 1] = 10_000                                        # tokens 18, 19 of sequence 0
    out = torch.full_like(q, 5.0)
    vdx.rope3d_append(q, k, k, cache, cu_of([2, 4]), c.kv_len, (100, 1, 1), q_out=out)
    with pytest.raises(vdx.VdxError, match="page index"):
        vdx.sync_check()
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    touched[good[1].long()[0], :4] = True
    assert torch.equal(c.k[~touched].view(torch.int16), k0[~touched].view(torch.int16))
    assert not bool((out[:2] == 5.0).all())                       # the queries have their positions all the same
    c.table.copy_(good)
    # kv_len smaller than the new tokens, a position past the grid, a cache index past the table
    for lens, grid, off in (([1, 4], (100, 1, 1), 0), ([20, 4], (2, 3, 3), 0), ([400, 4], (1000, 1, 1), 0), ([20, 4], (100, 1, 1), -19)):
        out.fill_(5.0)
        vdx.rope3d_append(q, k, k, cache, cu_of([2, 4]), torch.tensor(lens, dtype=torch.int32, device="cuda"), grid, q_out=out,
                          pos_offset=torch.tensor([off, 0], dtype=torch.int32, device="cuda"))
        with pytest.raises(vdx.VdxError, match="appended token"):
            vdx.sync_check()
        assert bool((out[0] == 5.0).all()) and not bool((out[2:] == 5.0).all())
    vdx.sync_check()


def test_append_nothing():
    c = Paged(torch.bfloat16, 64, 1, 16, [4], seed=14)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    r = vdx.rope3d_append(e, e, e, vdx.PagedKV(c.k, c.v, c.table), cu_of([0]), c.kv_len, (9, 1, 1))
    assert r.shape == e.shape
    vdx.rope3d_append(None, e, e, vdx.PagedKV(c.k, c.v, c.table), cu_of([0]), c.kv_len, (9, 1, 1))
    vdx.sync_check()


# ------------------------------------------------------------------------------------ paged attention
def _paged_case(dtype, d, Hq, Hkv, page, news, lens, block, order="token", seed=20, gain=1.5, pad=2, **kw):
    dt = DT[dtype]
    c = Paged(dt, d, Hkv, page, lens, seed=seed, order=order, **kw)
    n = sum(news)
    wide = _rand((n + pad, Hq + 2, d), dt, seed + 1, gain)
    q = wide[:, 1:Hq + 1]                                           # strided, like a slice of a projection
    out = torch.full((n + pad, Hq, d), 9.0, dtype=dt, device="cuda")
    lse = torch.full((Hq, n + pad), 7.0, device="cuda")
    return dt, c, q, out, lse


def _check_paged(c, q, out, lse, news, lens, block, dt, scale=None):
    at = 0
    for s, (m, length) in enumerate(zip(news, lens)):
        k, v = c.get(s, length)
        ref = attend(q[at:at + m], k, v, limits(m, length, block), scale)
        check_attention(out[at:at + m], lse[:, at:at + m], ref, dt, f"sequence {s}: {m} of {length}")
        at += m
    assert bool((out[at:] == 9.0).all()) and bool((lse[:, at:] == 7.0).all())   # rows behind the last sequence


PAGED = [
    # single tokens: lengths around the 16-key blocks, the pages and the splits; one sequence without rows, one without keys
    ("bf16", 128, 12, 12, 16, [1, 1, 1, 0, 1, 1], [1, 15, 16, 40, 17, 2000], 0),
    ("bf16", 128, 40, 8, 64, [1, 1, 1], [5000, 63, 64], 1),
    ("fp16", 64, 12, 1, 32, [1, 1, 0], [777, 33, 0], 0),
    ("fp16", 128, 4, 4, 200, [1, 1], [199, 4001], 1),
    ("bf16", 64, 33, 1, 16, [1, 2], [100, 50], 1),
    # few heads over long caches: many splits, joined through the workspace
    ("bf16", 128, 4, 1, 64, [1, 2, 1], [20000, 9001, 3], 1),
    ("fp16", 64, 2, 2, 200, [3, 0, 1], [30011, 5, 0], 0),
    # short chunks
    ("bf16", 128, 6, 2, 128, [5, 3, 8], [5, 300, 1029], 1),
    ("fp16", 64, 8, 8, 16, [16, 7], [16, 100], 3),
    # chunks of a tile and more, ragged, ends inside tiles and pages
    ("bf16", 128, 3, 3, 64, [128, 1, 300, 0, 65], [128, 700, 301, 64, 65], 1),
    ("bf16", 128, 2, 1, 130, [257, 100], [513, 100], 100),
    ("fp16", 64, 12, 4, 16, [200, 90, 1], [1000, 90, 333], 1),
    ("fp16", 128, 5, 1, 32, [150, 64], [150, 2100], 64),
    ("bf16", 64, 4, 4, 200, [400, 33], [999, 33], 0),
    ("bf16", 128, 2, 2, 1560, [1560, 390], [4680, 1950], 1560),
    ("bf16", 128, 64, 1, 16, [9, 2], [200, 2], 1),
    ("fp16", 128, 128, 1, 128, [3], [150], 1),
    ("bf16", 128, 1, 1, 128, [2048], [2048], 1),
    # more units of work than multiprocessors, of very different lengths
    ("bf16", 128, 12, 4, 64, [1, 300, 0, 77, 500, 33, 257, 2, 128, 90, 400, 5], [900, 300, 10, 1077, 500, 40, 600, 3, 129, 2000, 411, 5], 1),
    ("fp16", 64, 8, 8, 200, [256, 40, 0, 1, 600, 100, 90, 300], [300, 40, 200, 401, 1000, 150, 2090, 300], 50),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"{c[0]}-d{c[1]}-{c[2]}over{c[3]}-page{c[4]}-{max(c[5])}of{max(c[6])}-block{c[7]}")
@pytest.mark.parametrize("order", ["token", "head"])
def test_paged_attention_matches_the_formula(case, order):
    dtype, d, Hq, Hkv, page, news, lens, block = case
    dt, c, q, out, lse = _paged_case(*case, order=order)
    o, l = vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of(news), c.kv_len, max_q=max(news), max_kv=max(lens),
                          causal_block=block, out=out, lse=lse)
    vdx.sync_check()
    assert o is out and l is lse
    _check_paged(c, q, out, lse, news, lens, block, dt)


@pytest.mark.parametrize("news,lens", [([1, 1], [900, 40]), ([70, 300], [900, 400])])
def test_paged_attention_with_default_bounds_and_no_lse(news, lens):
    dt, c, q, out, lse = _paged_case("bf16", 128, 4, 2, 32, news, lens, 1, width=80)
    cache, cu = vdx.PagedKV(c.k, c.v, c.table), cu_of(news)
    vdx.paged_attn(q, cache, cu, c.kv_len, causal_block=1, out=out, lse=lse)
    ws = torch.empty(vdx.paged_attn_workspace_bytes(q, cache, cu, c.kv_len, max(news), max(lens)) + 16, dtype=torch.uint8, device="cuda")
    o2, none = vdx.paged_attn(q, cache, cu, c.kv_len, max(news), max(lens), causal_block=1, return_lse=False, workspace=ws)
    vdx.sync_check()
    assert none is None
    _check_paged(c, q, out, lse, news, lens, 1, dt)
    at = 0
    for s, (m, length) in enumerate(zip(news, lens)):
        k, v = c.get(s, length)
        ref = attend(q[at:at + m], k, v, limits(m, length, 1))
        check_attention(o2[at:at + m], ref[1].float(), ref, dt)
        at += m


@pytest.mark.parametrize("n", [3, 40, 300])
@pytest.mark.parametrize("block", [1, 4])
def test_rows_before_the_first_key_see_nothing(n, block):
    # fewer keys than new tokens: the first rows stand at negative positions
    length = n - 2
    dt, c, q, out, lse = _paged_case("bf16", 128, 2, 2, 16, [n], [length], block, width=30)
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of([n]), c.kv_len, max_q=n, max_kv=max(length, 1), causal_block=block,
                   out=out, lse=lse)
    vdx.sync_check()
    assert bool((out[:2] == 0).all()) and bool((lse[:, :2] == -math.inf).all())
    _check_paged(c, q, out, lse, [n], [length], block, dt)


def test_a_busy_sequence_among_many_idle_ones():
    # most units of work have no rows or no keys: a multiprocessor meets long runs of them between two with work
    S, dt = 700, torch.bfloat16
    news = [0] * S
    for s in (0, 1, 333, 334, 699):
        news[s] = 300
    lens = [n + 50 if n else (16 if s % 3 else 0) for s, n in enumerate(news)]
    lens[334] = 300
    dt, c, q, out, lse = _paged_case("bf16", 128, 4, 2, 16, news, lens, 1)
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of(news), c.kv_len, max_q=300, max_kv=350, causal_block=1, out=out, lse=lse)
    vdx.sync_check()
    _check_paged(c, q, out, lse, news, lens, 1, dt)


def test_cross_attention_with_whole_batch_entries_without_keys():
    q = _rand((6, 9000, 4, 128), torch.bfloat16, 90, 1.5)
    k, v = (_rand((6, 200, 4, 128), torch.bfloat16, s) for s in (91, 92))
    lens = [200, 0, 0, 0, 0, 70]
    out, lse = vdx.cross_attn(q, k, v, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    vdx.sync_check()
    for b, n in enumerate(lens):
        ref = attend(q[b], k[b, :n], v[b, :n], torch.full((9000,), n, device="cuda"))
        check_attention(out[b], lse[b], ref, torch.bfloat16, f"entry {b}")


@pytest.mark.parametrize("n", [2, 200])
def test_rows_with_no_keys_at_all(n):
    dt, c, q, out, lse = _paged_case("fp16", 64, 4, 4, 16, [n, n], [0, 30 if n < 30 else n], 0, width=20)
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of([n, n]), c.kv_len, max_q=n, causal_block=0, out=out, lse=lse)
    vdx.sync_check()
    assert bool((out[:n] == 0).all()) and bool((lse[:, :n] == -math.inf).all())
    _check_paged(c, q, out, lse, [n, n], [0, 30 if n < 30 else n], 0, dt)


@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_along_the_keys(n, rising):
    # the running maximum moves in every tile, or never again after the first
    length = 1500
    dt, c, q, out, lse = _paged_case("bf16", 128, 2, 2, 64, [n], [length], 0)
    k, v = c.get(0)
    ramp = torch.linspace(0.0, 60.0, length, device="cuda") * (1 if rising else -1)
    k = (k.float() * 0.2 + ramp[:, None, None] / 128 ** 0.5).to(dt)
    c.put(0, k, v)
    q.copy_((q.float() * 0.2 + 1.0).to(dt))
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of([n]), c.kv_len, max_q=n, max_kv=length, out=out, lse=lse)
    vdx.sync_check()
    _check_paged(c, q, out, lse, [n], [length], 0, dt)


@pytest.mark.parametrize("n", [1, 200])
def test_very_negative_scores_keep_their_weights(n):
    # all scores near -400: exponentials against zero would vanish
    dt, c, q, out, lse = _paged_case("bf16", 128, 1, 1, 16, [n], [300], 0)
    k, v = c.get(0)
    c.put(0, (k.float() * 0.3 - 6.0).to(dt), v)
    q.copy_((q.float() * 0.1 + 6.0).to(dt))
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of([n]), c.kv_len, max_q=n, max_kv=300, out=out, lse=lse)
    vdx.sync_check()
    _check_paged(c, q, out, lse, [n], [300], 0, dt)


@pytest.mark.parametrize("n", [1, 200])
def test_masked_keys_may_be_infinite(n):
    # a future key of NaN or infinity changes nothing for the rows before it; its value stays finite
    length = 400
    dt, c, q, out, lse = _paged_case("bf16", 128, 2, 2, 16, [n], [length], 1)
    k, v = c.get(0)
    bad = k.clone()
    bad[-1] = math.inf
    bad[-1, :, ::2] = math.nan
    c.put(0, bad, v)
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of([n]), c.kv_len, max_q=n, max_kv=length, causal_block=1, out=out, lse=lse)
    vdx.sync_check()
    assert bool(torch.isnan(out[n - 1]).all())
    if n > 1:
        ref = attend(q[:n - 1], k, v, limits(n, length, 1)[:-1])
        check_attention(out[:n - 1], lse[:, :n - 1], ref, dt)


@pytest.mark.parametrize("n", [1, 200])
def test_bad_pages_and_lengths_are_reported(n):
    news, lens = [n, n], [250, 300]
    dt, c, q, out, lse = _paged_case("bf16", 128, 2, 2, 16, news, lens, 0)
    cache = vdx.PagedKV(c.k, c.v, c.table)
    good = c.table.clone()
    for bad in (-1, c.k.shape[0], 1 << 30):
        c.table[0, 3] = bad
        vdx.paged_attn(q, cache, cu_of(news), c.kv_len, max_q=n, max_kv=300, out=out, lse=lse)
        with pytest.raises(vdx.VdxError, match="page index"):
            vdx.sync_check()
        k, v = c.get(1, 300)                                        # the other sequence is right
        check_attention(out[n:2 * n], lse[:, n:2 * n], attend(q[n:2 * n], k, v, limits(n, 300, 0)), dt)
        c.table.copy_(good)
    out.fill_(9.0)
    for kw in (dict(max_q=n, max_kv=299), dict(max_q=n, max_kv=300, kv_len=torch.tensor([250, 100000], dtype=torch.int32, device="cuda")),
               dict(max_q=n, max_kv=300, kv_len=torch.tensor([250, -3], dtype=torch.int32, device="cuda")),
               dict(max_q=n, max_kv=300, cu=torch.tensor([0, n, 100000], dtype=torch.int32, device="cuda")),
               dict(max_q=n, max_kv=300, cu=torch.tensor([0, n, n - 1], dtype=torch.int32, device="cuda"))):
        cu, kl = kw.pop("cu", cu_of(news)), kw.pop("kv_len", c.kv_len)
        vdx.paged_attn(q, cache, cu, kl, out=out, lse=lse, **kw)
        with pytest.raises(vdx.VdxError, match="clamped"):
            vdx.sync_check()
        k, v = c.get(0, 250)
        check_attention(out[:n], lse[:, :n], attend(q[:n], k, v, limits(n, 250, 0)), dt)
    if n > 1:
        vdx.paged_attn(q, cache, cu_of(news), c.kv_len, max_q=n - 1, max_kv=300, out=out, lse=lse)
        with pytest.raises(vdx.VdxError, match="clamped"):
            vdx.sync_check()
    vdx.paged_attn(q, cache, cu_of(news), c.kv_len, max_q=n, max_kv=300, out=out, lse=lse)
    vdx.sync_check()


def test_shared_prefix_pages_and_a_repeated_page():
    # two sequences read the same pages; a third names one page twice
    dt, c, q, out, lse = _paged_case("bf16", 128, 2, 2, 16, [1, 1, 1], [64, 64, 32], 0, width=4)
    c.table[1] = c.table[0]
    c.table[2, :2] = c.table[0, 0]
    vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of([1, 1, 1]), c.kv_len, max_q=1, max_kv=64, out=out, lse=lse)
    vdx.sync_check()
    _check_paged(c, q, out, lse, [1, 1, 1], [64, 64, 32], 0, dt)


# ------------------------------------------------------------------------------------ cross attention
CROSS = [
    ("fp16", 64, 1, 192, 77, 4, 4, None),
    ("bf16", 128, 2, 1000, 512, 3, 3, [512, 131]),
    ("bf16", 128, 3, 1, 257, 12, 4, [257, 0, 1]),
    ("bf16", 128, 2, 300, 1, 2, 2, None),
    ("fp16", 128, 2, 129, 128, 5, 5, [127, 128]),
    ("bf16", 64, 1, 513, 130, 8, 2, None),
    ("fp16", 64, 2, 20, 7, 6, 6, [7, 3]),
    ("bf16", 128, 1, 256, 1024, 40, 8, None),
    ("bf16", 128, 4, 700, 129, 1, 1, [129, 128, 0, 64]),
    # more units of work than multiprocessors: each takes several in turn, some without keys
    ("bf16", 128, 3, 2000, 300, 20, 20, [300, 0, 130]),
    ("fp16", 64, 5, 1100, 700, 16, 16, [1, 700, 0, 129, 640]),
]


@pytest.mark.parametrize("case", CROSS, ids=lambda c: f"{c[0]}-d{c[1]}-{c[3]}over{c[4]}-heads{c[5]}over{c[6]}{'-ragged' if c[7] else ''}")
def test_cross_attention_matches_the_formula(case):
    dtype, d, Bn, N, M, Hq, Hkv, lens = case
    dt = DT[dtype]
    q = _rand((Bn, N, Hq, d), dt, 30, 1.5)
    kv = _rand((Bn, M, 2, Hkv, d), dt, 31)                           # one projection's output
    k, v = kv[:, :, 0], kv[:, :, 1]
    kl = None
    if lens:
        kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            kv[b, n:] = math.nan                                       # padding is never used
    out, lse = vdx.cross_attn(q, k, v, kv_len=kl)
    vdx.sync_check()
    for b in range(Bn):
        n = lens[b] if lens else M
        ref = attend(q[b], k[b, :n], v[b, :n], torch.full((N,), n, device="cuda"))
        check_attention(out[b], lse[b], ref, dt, f"entry {b}")


@pytest.mark.parametrize("N", [2, 300])
def test_cross_attention_shares_broadcast_inputs(N):
    q = _rand((3, N, 2, 128), torch.bfloat16, 32)
    k, v = (_rand((1, 200, 2, 128), torch.bfloat16, s) for s in (33, 34))
    a, la = vdx.cross_attn(q, k.expand(3, -1, -1, -1), v.expand(3, -1, -1, -1), scale=0.05)
    b, lb = vdx.cross_attn(q, k.repeat(3, 1, 1, 1), v.repeat(3, 1, 1, 1), scale=0.05)
    c, lc = vdx.cross_attn(q[:1].expand(3, -1, -1, -1), k.expand(3, -1, -1, -1), v.expand(3, -1, -1, -1), scale=0.05)
    vdx.sync_check()
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert torch.equal(c[2], a[0]) and torch.equal(lc[1], la[0])
    ref = attend(q[1], k[0], v[0], torch.full((N,), 200, device="cuda"), 0.05)
    check_attention(a[1], la[1], ref, torch.bfloat16)


@pytest.mark.parametrize("N", [2, 300])
def test_cross_attention_of_head_major_tensors_and_no_keys(N):
    q = _rand((2, 3, N, 64), torch.float16, 35).transpose(1, 2)
    k, v = (_rand((2, 3, 50, 64), torch.float16, s).transpose(1, 2) for s in (36, 37))
    out, lse = vdx.cross_attn(q, k, v)
    e = k[:, :0]
    zero, none = vdx.cross_attn(q, e, e)
    got = vdx.cross_attn(q[:, :0], k, v)
    vdx.sync_check()
    for b in range(2):
        check_attention(out[b], lse[b], attend(q[b], k[b], v[b], torch.full((N,), 50, device="cuda")), torch.float16)
    assert bool((zero == 0).all()) and bool((none == -math.inf).all())
    assert got[0].shape == (2, 0, 3, 64) and got[1].shape == (2, 3, 0)


def test_cross_attention_reports_lengths_past_the_keys():
    q, k = _rand((2, 5, 1, 64), torch.bfloat16, 38), _rand((2, 9, 1, 64), torch.bfloat16, 39)
    out, lse = vdx.cross_attn(q, k, k, kv_len=torch.tensor([10, -1], dtype=torch.int32, device="cuda"))
    with pytest.raises(vdx.VdxError, match="clamped"):
        vdx.sync_check()
    check_attention(out[0], lse[0], attend(q[0], k[0], k[0], torch.full((5,), 9, device="cuda")), torch.bfloat16)
    assert bool((out[1] == 0).all())


# ------------------------------------------------------------------------------------ together
def _stream_block(steps, dt, Hq, Hkv, d, page, grid, chunk, wq, wk, cache, table, xs, text, graph=None):
    """Frame-causal generation: per chunk, append, attend over the cache, attend to the text."""
    outs = []
    for t in range(steps):
        q, k, v = xs[t][:, :Hq], xs[t][:, Hq:Hq + Hkv], xs[t][:, Hq + Hkv:]
        kv_len = torch.tensor([chunk * (t + 1)] * 2, dtype=torch.int32, device="cuda")
        qr = vdx.rope3d_append(q, k, v, cache, cu_of([chunk, chunk]), kv_len, grid, SECTIONS[d], q_norm=wq, k_norm=wk)
        o, _ = vdx.paged_attn(qr, cache, cu_of([chunk, chunk]), kv_len, max_q=chunk, max_kv=chunk * (t + 1), causal_block=chunk)
        c, _ = vdx.cross_attn(o.view(2, chunk, Hq, d), text[0], text[1])
        outs.append((qr, o, c))
    return outs


def test_a_streaming_block_equals_full_attention():
    # chunk by chunk over the cache = frame-causal attention over the whole sequence in 64 bits
    dt, Hq, Hkv, d, page, chunk, steps = torch.bfloat16, 4, 2, 128, 200, 6 * 9, 4
    grid = (steps, 6, 9)
    wq, wk = _rand((d,), dt, 40), _rand((d,), dt, 41)
    xs = [_rand((2 * chunk, Hq + 2 * Hkv, d), dt, 42 + t) for t in range(steps)]
    text = [_rand((2, 33, Hkv, d), dt, s) for s in (50, 51)]
    pages = 2 * -(-chunk * steps // page)
    k_cache, v_cache = (torch.full((pages, page, Hkv, d), math.nan, dtype=dt, device="cuda") for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).view(2, -1).contiguous()
    cache = vdx.PagedKV(k_cache, v_cache, table)
    outs = _stream_block(steps, dt, Hq, Hkv, d, page, grid, chunk, wq, wk, cache, table, xs, text)
    vdx.sync_check()
    for s in range(2):
        rows = [x[s * chunk:(s + 1) * chunk] for x in xs]
        full = torch.cat(rows)
        pos = torch.arange(chunk * steps, device="cuda")
        k_ref = rotate(full[:, Hq:Hq + Hkv], pos, grid, SECTIONS[d], 10000.0, wk, 1e-6)
        q_ref = rotate(full[:, :Hq], pos, grid, SECTIONS[d], 10000.0, wq, 1e-6)
        # the cache and the rotated queries hold one rounding; attention is then checked on what they hold
        slots = (table[s].long()[pos // page], pos % page)
        kc, vc = k_cache[slots], v_cache[slots]
        assert bool(((kc.double() - k_ref).abs() <= rotate_bound(k_ref, dt)).all()) and torch.equal(vc, full[:, Hq + Hkv:])
        for t, (qr, o, c) in enumerate(outs):
            part = slice(s * chunk, (s + 1) * chunk)
            qt = q_ref[t * chunk:(t + 1) * chunk]
            assert bool(((qr[part].double() - qt).abs() <= rotate_bound(qt, dt)).all())
            length = chunk * (t + 1)
            ref = attend(qr[part], kc[:length], vc[:length], torch.full((chunk,), length, device="cuda"))
            check_attention(o[part], ref[1].float(), ref, dt, f"sequence {s} chunk {t}")
            ref = attend(o[part], text[0][s], text[1][s], torch.full((chunk,), 33, device="cuda"))
            check_attention(c[s], ref[1].float(), ref, dt, f"text {s} chunk {t}")


def test_a_captured_step_replays_with_new_lengths():
    # one graph of append + attention + cross attention; lengths, pages and inputs change between replays
    dt, H, d, page = torch.bfloat16, 4, 128, 16
    c = Paged(dt, d, H, page, [500, 900], seed=60, width=64, spare=10)
    cache = vdx.PagedKV(c.k, c.v, c.table)
    x = _rand((2, 3 * H, d), dt, 61)
    text = _rand((2, 40, H, d), dt, 62)
    cu = cu_of([1, 1])

    def step():
        q = vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], cache, cu, c.kv_len, (2000, 1, 1))
        o, l = vdx.paged_attn(q, cache, cu, c.kv_len, max_q=1, max_kv=1000)
        y, _ = vdx.cross_attn(o.view(2, 1, H, d), text, text)
        return q, o, l, y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, results = [], []
    for _ in range(2):                                                # two graphs in flight do not share scratch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(step())
        graphs.append(g)
    for lens in ([500, 900], [37, 901], [501, 17]):                     # every key below them was written once
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        x.copy_(_rand((2, 3 * H, d), dt, sum(lens)))
        for (q, o, l, y), g in zip(results, graphs):
            o.zero_()
            g.replay()
        eager = step()
        vdx.sync_check()
        for r in results:
            for a, b in zip(r, eager):
                assert torch.equal(a, b)
        for s, n in enumerate(lens):
            k, v = c.get(s, n)
            check_attention(o[s:s + 1], l[:, s:s + 1], attend(q[s:s + 1], k, v, limits(1, n, 0)), dt, f"{s} {n}")
    ga, gb = torch.cuda.Stream(), torch.cuda.Stream()
    want = step()
    torch.cuda.synchronize()
    for s, g in ((ga, graphs[0]), (gb, graphs[1])):
        with torch.cuda.stream(s):
            for _ in range(20):
                g.replay()
    torch.cuda.synchronize()
    for r in results:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


def test_a_captured_chunk_replays_with_new_lengths():
    # the tile kernel and its joined splits in a graph: chunk lengths, cached lengths and inputs change between replays
    dt, H, d, page, S = torch.bfloat16, 4, 128, 64, 3
    c = Paged(dt, d, H, page, [3000, 2500, 700], seed=95, width=64)
    cache = vdx.PagedKV(c.k, c.v, c.table)
    q = _rand((600, H, d), dt, 96)
    text = _rand((S, 150, H, d), dt, 97)
    cu = cu_of([200, 200, 200])
    out, lse = torch.full_like(q, 9.0), torch.full((H, 600), 7.0, device="cuda")

    def step():
        vdx.paged_attn(q, cache, cu, c.kv_len, max_q=300, max_kv=3000, causal_block=1, out=out, lse=lse)
        return vdx.cross_attn(q.view(S, 200, H, d), text, text)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, ly = step()
    for news, lens in (([200, 200, 200], [3000, 2500, 700]), ([300, 0, 150], [2999, 40, 150]), ([1, 299, 300], [64, 299, 700])):
        cu.copy_(cu_of(news))
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(_rand((600, H, d), dt, sum(news)))
        out.fill_(9.0)
        lse.fill_(7.0)
        g.replay()
        vdx.sync_check()
        _check_paged(c, q, out, lse, news, lens, 1, dt)
        for b in range(S):
            ref = attend(q.view(S, 200, H, d)[b], text[b], text[b], torch.full((200,), 150, device="cuda"))
            check_attention(y[b], ly[b], ref, dt, f"text {b}")


@pytest.mark.parametrize("n", [1, 300])
def test_calls_on_a_side_stream_and_repeated_calls_are_bit_identical(n):
    dt, c, q, out, lse = _paged_case("bf16", 128, 4, 4, 64, [n, n], [3000, 777], 0)
    cache, cu = vdx.PagedKV(c.k, c.v, c.table), cu_of([n, n])
    a, la = vdx.paged_attn(q, cache, cu, c.kv_len, max_q=n, max_kv=3000, out=out.clone(), lse=lse.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [vdx.paged_attn(q, cache, cu, c.kv_len, max_q=n, max_kv=3000, out=out.clone(), lse=lse.clone(), stream=s)
            for s in (None, side, torch.cuda.current_stream())]
    own = vdx.paged_attn(q, cache, cu, c.kv_len, max_q=n, max_kv=3000, stream=side)
    vdx.sync_check(side)
    vdx.sync_check()
    for o, l in outs:
        assert torch.equal(a, o) and torch.equal(la, l)
    assert torch.equal(own[0][:2 * n], a[:2 * n])


def test_two_threads_on_two_streams_at_once():
    import threading
    dt, rows, keys = torch.bfloat16, (1, 40), (9000, 700)             # joined splits; tiles
    cases = [(_rand((1, n, 4, 128), dt, 80 + n), _rand((1, m, 4, 128), dt, 90 + n)) for n, m in zip(rows, keys)]
    want = [vdx.cross_attn(q, k, k) for q, k in cases]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            q, k = cases[i]
            for j in range(30):
                if j % 3 == 2:
                    with pytest.raises(vdx.VdxError, match="must have"):
                        vdx.cross_attn(q, k[0], k, stream=stream)
                got[i].append(vdx.cross_attn(q, k, k, stream=stream))
            stream.synchronize()
        except BaseException as e:                                     # a failed assertion must reach the test
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    vdx.sync_check()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 30
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])


def test_calls_keep_no_references_and_no_memory():
    import sys
    dt = torch.bfloat16
    c = Paged(dt, 128, 2, 16, [40, 9], seed=66)
    cache, x, w = vdx.PagedKV(c.k, c.v, c.table), _rand((2, 2, 128), dt, 67), _rand((128,), dt, 68)
    cu, text = cu_of([1, 1]), _rand((1, 50, 2, 128), dt, 69)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    grid, q_out, out = (50, 1, 1), torch.empty_like(x), torch.empty_like(x)
    kept = [c.k, c.v, c.table, c.kv_len, x, w, cu, text, none, grid, q_out, out]

    def calls():
        vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, grid, q_norm=w, k_norm=w)
        vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, list(grid), q_out=q_out)
        assert vdx.rope3d_append(None, x, x, cache, cu, c.kv_len, grid) is None
        assert vdx.paged_attn(x, cache, cu, c.kv_len, out=out)[0] is out
        assert vdx.paged_attn(x, cache, cu, c.kv_len, return_lse=False)[1] is None
        vdx.cross_attn(text, text, text, kv_len=none)
        with pytest.raises(vdx.VdxError):
            vdx.paged_attn(x, cache, cu[:2], c.kv_len)
        with pytest.raises(vdx.VdxError):
            vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, 1))
        with pytest.raises(TypeError):
            vdx.cross_attn(text, text, text, scale="x")
        with pytest.raises(vdx.VdxError):
            vdx.cross_attn(text, text, text, out=text[:, :9])

    calls()
    torch.cuda.synchronize()
    before, memory = [sys.getrefcount(t) for t in kept], torch.cuda.memory_allocated()
    for _ in range(20):
        calls()
    torch.cuda.synchronize()
    assert [sys.getrefcount(t) for t in kept] == before and torch.cuda.memory_allocated() == memory


def test_what_the_calls_refuse_of_tensors():
    dt = torch.bfloat16
    c = Paged(dt, 128, 2, 16, [40, 9], seed=70)
    cache, x, cu = vdx.PagedKV(c.k, c.v, c.table), _rand((2, 2, 128), dt, 71), cu_of([1, 1])
    text = _rand((1, 50, 2, 128), dt, 72)
    grad = x.clone().requires_grad_()
    refused = [
        lambda: vdx.paged_attn(grad, cache, cu, c.kv_len),
        lambda: vdx.paged_attn(x.float(), cache, cu, c.kv_len),
        lambda: vdx.paged_attn(x.cpu(), cache, cu, c.kv_len),
        lambda: vdx.paged_attn(None, cache, cu, c.kv_len),
        lambda: vdx.paged_attn(x[0], cache, cu, c.kv_len),
        lambda: vdx.paged_attn(x[..., ::2], cache, cu, c.kv_len),
        lambda: vdx.paged_attn(x, cache, None, c.kv_len),
        lambda: vdx.paged_attn(x, cache, cu.long(), c.kv_len),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len.cpu()),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len, max_q=-1),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len, max_kv=2 ** 31),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len, out=x),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len, lse=torch.empty(2, 2, device="cuda", dtype=torch.float64)),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len, lse=torch.empty(3, 2, device="cuda")),
        lambda: vdx.paged_attn(x, cache, cu, c.kv_len, workspace=torch.empty(64)),
        lambda: vdx.paged_attn(x, vdx.PagedKV(c.k, c.v[:1], c.table), cu, c.kv_len),
        lambda: vdx.paged_attn(x, vdx.PagedKV(c.k, c.v.half(), c.table), cu, c.kv_len),
        lambda: vdx.paged_attn(x, vdx.PagedKV(c.k, c.v, c.table.long()), cu, c.kv_len),
        lambda: vdx.paged_attn(x, vdx.PagedKV(c.k, c.v, c.table[0]), cu, c.kv_len),
        lambda: vdx.paged_attn_workspace_bytes(x, vdx.PagedKV(c.k, c.v, None), cu, c.kv_len),
        lambda: vdx.rope3d_append(x, x, x[:1], cache, cu, c.kv_len, (50, 1, 1)),
        lambda: vdx.rope3d_append(x[:1], x, x, cache, cu, c.kv_len, (50, 1, 1)),
        lambda: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, 1, 1), q_norm=x[0, 0, :64]),
        lambda: vdx.rope3d_append(None, x, x, cache, cu, c.kv_len, (50, 1, 1), q_out=x),
        lambda: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, 1, 1), q_out=torch.empty_like(x)[:1]),
        lambda: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, -1, 1)),
        lambda: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, 1, 1), sections=(0, 0)),
        lambda: vdx.cross_attn(text, text[..., :64], text[..., :64]),
        lambda: vdx.cross_attn(text, text, text[:, :9]),
        lambda: vdx.cross_attn(text.double(), text.double(), text.double()),
        lambda: vdx.cross_attn(text.to_sparse(), text, text),
        lambda: vdx.cross_attn_workspace_bytes(text, text, text.half()),
    ]
    for i, f in enumerate(refused):
        with pytest.raises(vdx.VdxError):
            f()
            pytest.fail(f"call {i} was taken")
    with torch.no_grad():
        vdx.paged_attn(grad, cache, cu, c.kv_len)


def test_a_row_of_nan_is_its_own_answer_only():
    # in each kernel: few rows, few rows over a long cache (joined), many rows
    dt = torch.float16
    for rows, keys, bad in ((3, 50, 1), (2, 9000, 0), (300, 400, 170)):
        q, k = _rand((1, rows, 2, 64), dt, 73), _rand((1, keys, 2, 64), dt, 74)
        # (the rows of a warp raise their running maxima together, by up to 2^8 late, so the other rows' last bits
        # may depend on this one; the bounds against the formula cover that)
        ref = attend(q[0], k[0], k[0], limits(rows, keys, 0))
        q2 = q.clone()
        q2[0, bad, 1, 5] = float("nan")
        got, gl = vdx.cross_attn(q2, k, k)
        assert bool(got[0, bad, 1].isnan().all()) and bool(gl[0, 1, bad].isnan())
        got[0, bad, 1], gl[0, 1, bad] = ref[0][bad, 1].to(dt), ref[1][1, bad].float()
        check_attention(got[0], gl[0], ref, dt, str(rows))


def test_cache_offsets_past_32_bits():
    # pages far enough apart that element offsets pass 2^31
    page, H, d = 1024, 8, 128
    pages = (1 << 31) // (page * H * d) + 3
    k = torch.empty((pages, page, H, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[pages - 1, 0], [pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    table[1, 1] = 1
    for n in (1, 140):
        x = _rand((2 * n, 3 * H, d), torch.bfloat16, 70)
        kv_len = torch.tensor([1100, 200], dtype=torch.int32, device="cuda")
        for s, length in ((0, 1100), (1, 200)):
            for i in range(2):
                k[table[s, i].long()] = _rand((page, H, d), torch.bfloat16, 71 + i + 2 * s)
                v[table[s, i].long()] = _rand((page, H, d), torch.bfloat16, 81 + i + 2 * s)
        cache = vdx.PagedKV(k, v, table)
        q = vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], cache, cu_of([n, n]), kv_len, (2000, 1, 1))
        out, lse = vdx.paged_attn(q, cache, cu_of([n, n]), kv_len, max_q=n, max_kv=1100, causal_block=1)
        vdx.sync_check()
        for s, length in ((0, 1100), (1, 200)):
            keys = torch.arange(length, device="cuda")
            kk, vv = (t[table[s].long()[keys // page], keys % page] for t in (k, v))
            ref = attend(q[s * n:(s + 1) * n], kk, vv, limits(n, length, 1))
            check_attention(out[s * n:(s + 1) * n], lse[:, s * n:(s + 1) * n], ref, torch.bfloat16)
            assert torch.equal(vv[-n:], x[s * n:(s + 1) * n, 2 * H:])
