"""The 8-bit paged cache: appending to it and attention over it, against the definition in 64 bits."""
import math

import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from kv8_ref import BLOCK, CODE, E_MAX, SCALE, Paged8, check_attention8, codes64, exps, half_step8, least_exponent, powers, round8
from streaming_ref import DT, SECTIONS, attend, cu_of, limits, rotate, rotate_bound

pytestmark = pytest.mark.gpu


def _rand(shape, dtype, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


# ------------------------------------------------------------------------------------------------ append
def _check_blocks(c, want_k, first_new, news):
    """Keys of every sequence against their 64-bit values want_k[s] [n, Hkv, d] and fp32 error err[s]: scales, codes of new
    tokens, codes of older ones in the first block."""
    for s, (x, slack, before) in enumerate(want_k):
        n, f = x.shape[0], first_new[s]
        a = f
        while a < f + n:
            page, slot = int(c.table[s, a // c.page]), a % c.page
            b = slot // BLOCK
            stop = min(f + n, a - slot + min(c.page, (b + 1) * BLOCK))
            val, sl = x[a - f:stop - f], slack[a - f:stop - f]
            lo, hi = least_exponent((val.abs() - sl).amax((0, 2)).clamp_min(0)), least_exponent((val.abs() + sl).amax((0, 2)))
            got = exps(c.k_scale)[page, b]
            if slot > b * BLOCK:
                old_e = exps(before.k_scale)[page, b]
                lo, hi = torch.maximum(lo, old_e), torch.maximum(hi, old_e)
                old = codes64(before.k[page, b * BLOCK:slot]) * powers(old_e - got)[None, :, None]
                assert torch.equal(codes64(c.k[page, b * BLOCK:slot]), round8(old)), (s, a)
            assert bool(((got >= lo) & (got <= hi)).all()), (s, a, got, lo, hi)
            unit = powers(got)[None, :, None]
            got_x = codes64(c.k[page, slot:slot + stop - a]) * unit
            bound = half_step8(val / unit) * unit * 1.0001 + sl
            err = (got_x - val).abs()
            assert bool((err <= bound).all()), (s, a, float((err / bound).max()))
            a = stop


APPEND = [
    # dtype, d, Hq, Hkv, page, new tokens, tokens before, grid, norm, order
    ("bf16", 128, 12, 12, 16, [1] * 9, [0, 1, 15, 16, 17, 31, 100, 255, 256], (999, 1, 1), True, "token"),
    ("bf16", 128, 4, 4, 128, [300, 45], [0, 77], (40, 3, 5), True, "token"),
    ("fp16", 64, 12, 4, 32, [1, 33, 0, 170, 15, 16, 17, 2], [5, 0, 40, 31, 1, 16, 15, 0], (500, 1, 1), False, "token"),
    ("fp16", 128, 4, 1, 200, [401, 1, 9], [190, 199, 200], (31, 5, 7), True, "head"),
    ("bf16", 64, 6, 3, 129, [260, 128, 1], [120, 1, 128], (10, 7, 9), False, "head"),
    ("bf16", 128, 40, 8, 1560, [1560, 3], [8, 1559], (9, 30, 52), True, "token"),
    ("bf16", 64, 2, 2, 64, [1], [0], (1, 1, 1), True, "token"),
]


@pytest.mark.parametrize("dtype,d,Hq,Hkv,page,news,ctxs,grid,norm,order", APPEND)
@pytest.mark.parametrize("gain", [1.0, 2.0 ** -9])
def test_append_matches_the_definition(dtype, d, Hq, Hkv, page, news, ctxs, grid, norm, order, gain):
    dt = DT[dtype]
    lens = [a + b for a, b in zip(news, ctxs)]
    c = Paged8(d, Hkv, page, ctxs, seed=3, order=order, width=-(-max(lens) // page) + 1, scale_order="page" if order == "head" else "head")
    # the pages of the new tokens: fresh ones
    free = [i for i in range(c.k.shape[0]) if i not in set(c.table[c.table >= 0].tolist())]
    need = sum(-(-n // page) for n in lens) + 2 - c.k.shape[0]
    if need > 0:
        def more(t, fill):
            shape = list(t.shape)
            shape[0] = need
            return torch.cat([t.view(torch.uint8), torch.full(shape, fill, dtype=torch.uint8, device="cuda")]).view(t.dtype)
        free += list(range(c.k.shape[0], c.k.shape[0] + need))
        c.k, c.v, c.k_scale, c.v_scale = more(c.k, 0x7f), more(c.v, 0x7f), more(c.k_scale, 0xff), more(c.v_scale, 0xff)
    for s, n in enumerate(lens):
        for i in range(-(-ctxs[s] // page), -(-n // page)):
            c.table[s, i] = free.pop()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rows = sum(news)
    qkv = _rand((rows + 3, Hq + 2 * Hkv, d), dt, 11, gain)
    qkv[:, :, 5] *= 6
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    qw, kw = (1 + 0.2 * _rand((d,), torch.float32, 12 + i) for i in range(2))
    qw, kw = (qw.to(dt), kw.to(dt)) if norm else (None, None)
    before, want = c.clone(), c.clone()
    got_q = vdx.rope3d_append(q, k, v, c.cache(vdx), cu_of(news), kv_len, grid, SECTIONS[d], 10000.0, q_norm=qw, k_norm=kw, eps=1e-6)
    vdx.sync_check()
    at, keys = 0, []
    for s, n in enumerate(news):
        pos = torch.arange(ctxs[s], lens[s], device="cuda")
        x = rotate(k[at:at + n], pos, grid, SECTIONS[d], 10000.0, kw, 1e-6)
        pair = torch.sqrt(x[..., 0::2] ** 2 + x[..., 1::2] ** 2).repeat_interleave(2, dim=-1)
        keys.append((x, 2.0 ** -19 * pair, before))
        ref_q = rotate(q[at:at + n], pos, grid, SECTIONS[d], 10000.0, qw, 1e-6)
        assert bool(((got_q[at:at + n].double() - ref_q).abs() <= rotate_bound(ref_q, dt)).all())
        want.put(want.v, want.v_scale, s, ctxs[s], v[at:at + n].double())
        at += n
    _check_blocks(c, keys, ctxs, news)
    # values are exact, and nothing else is touched
    assert torch.equal(c.v.view(torch.uint8), want.v.view(torch.uint8)) and torch.equal(c.v_scale.view(torch.uint8), want.v_scale.view(torch.uint8))
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    scaled = torch.zeros(c.k_scale.shape[:2], dtype=torch.bool, device="cuda")
    for s, n in enumerate(news):
        page_, slot = c.spots(s, ctxs[s], n)
        scaled[page_, slot // BLOCK] = True
        first = ctxs[s] - ctxs[s] % page % BLOCK if n else ctxs[s]
        page_, slot = c.spots(s, first, lens[s] - first)
        touched[page_, slot] = True
    assert torch.equal(c.k.view(torch.uint8)[~touched], before.k.view(torch.uint8)[~touched])
    assert torch.equal(c.k_scale.view(torch.uint8)[~scaled], before.k_scale.view(torch.uint8)[~scaled])


@pytest.mark.parametrize("dtype,d,norm", [("bf16", 128, True), ("fp16", 64, False)])
def test_a_chunk_and_its_pieces_give_the_same_bits(dtype, d, norm):
    # blocks that are appended whole have one scale, however many tokens the call has beside them
    dt, H, n = DT[dtype], 12, 1104
    q, k, v = (_rand((n, H, d), dt, 60 + i) for i in range(3))
    w = (1 + 0.1 * _rand((d,), torch.float32, 63)).to(dt) if norm else None
    got = []
    for pieces in ([1104], [800, 304], [320, 320, 320, 144], [16] * 69):
        c = Paged8(d, H, 128, [0], seed=1, width=9)
        c.k, c.v = (torch.zeros(9, 128, H, d, dtype=torch.uint8, device="cuda").view(c.k.dtype) for _ in range(2))
        c.k_scale, c.v_scale = (torch.zeros(9, 8, H, dtype=torch.uint8, device="cuda").view(c.k_scale.dtype) for _ in range(2))
        c.table = torch.arange(9, dtype=torch.int32, device="cuda").view(1, 9)
        at, qs = 0, []
        for m in pieces:
            kv_len = torch.tensor([at + m], dtype=torch.int32, device="cuda")
            qs.append(vdx.rope3d_append(q[at:at + m], k[at:at + m], v[at:at + m], c.cache(vdx), cu_of([m]), kv_len, (99, 6, 7), q_norm=w, k_norm=w))
            at += m
        vdx.sync_check()
        got.append([torch.cat(qs)] + [x.view(torch.uint8) for x in (c.k, c.v, c.k_scale, c.v_scale)])
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64)])
def test_a_scale_grows_and_older_codes_are_rounded_again(dtype, d):
    # one token at a time, each larger than the one before; then smaller ones, which leave the scale alone
    dt, H = DT[dtype], 3
    c = Paged8(d, H, 16, [0], seed=1, width=2)
    c.table[0] = torch.tensor([2, 0], dtype=torch.int32)
    want = c.clone()
    for i in range(20):
        x = _rand((1, H, d), dt, 50 + i, 2.0 ** (i - 8 if i < 12 else -4))
        vdx.rope3d_append(None, x, x, c.cache(vdx), cu_of([1]), torch.tensor([i + 1], dtype=torch.int32, device="cuda"), (99, 1, 1))
        want.put(want.v, want.v_scale, 0, i, x.double())
    vdx.sync_check()
    assert torch.equal(c.v.view(torch.uint8), want.v.view(torch.uint8)) and torch.equal(c.v_scale.view(torch.uint8), want.v_scale.view(torch.uint8))


def test_zeros_tiny_huge_and_nan_values():
    d, H = 128, 2
    c = Paged8(d, H, 16, [0], seed=1, width=4)
    c.table[0] = torch.tensor([0, 1, 2, 0], dtype=torch.int32)
    x = torch.zeros(48, H, d, dtype=torch.bfloat16, device="cuda")
    x[16:32, 0] = 2.0 ** -30                    # below every step of the least scale
    x[16:32, 1] = 2.0 ** -25 * 1.5              # rounds to its least number
    x[32, 0, 0] = math.nan
    x[33, 0, 1] = 2.0
    x[32, 1] = 57344.0
    args = (c.cache(vdx), cu_of([48]), torch.tensor([48], dtype=torch.int32, device="cuda"), (99, 1, 1))
    vdx.rope3d_append(None, torch.zeros_like(x), x, *args)
    vdx.sync_check()
    e = exps(c.v_scale)[:3, 0]
    assert e.tolist() == [[-15, -15], [-15, -15], [-7, 7]]
    v = codes64(c.v)
    assert bool((v[:2, :, 0] == 0).all()) and bool((v[1, :, 1] == 2.0 ** -9).all())
    assert bool(torch.isnan(v[2, 0, 0, 0])) and float(v[2, 1, 0, 1]) == 256.0 and bool((v[2, 0, 1] == 448).all())
    x[40, 1, 3] = -65536.0
    x[41, 1, 3] = math.inf
    vdx.rope3d_append(None, torch.zeros_like(x), x, *args)
    with pytest.raises(vdx.VdxError, match="clamped") as err:
        vdx.sync_check()
    assert err.value.status == 6
    v = codes64(c.v)
    assert float(v[2, 8, 1, 3]) == -448 and float(v[2, 9, 1, 3]) == 448 and int(exps(c.v_scale)[2, 0, 1]) == E_MAX


def test_append8_skips_and_reports_what_has_no_place():
    d, H, dt = 64, 2, torch.bfloat16
    c = Paged8(d, H, 16, [0, 0, 0, 0], seed=1, spare=8, width=2)
    c.table[:] = torch.tensor([[0, 1], [99, 2], [3, 4], [5, 6]], dtype=torch.int32)
    x = _rand((41, H, d), dt, 5)
    # within the table and partly past it; a bad first page; before the cache; past the grid
    news, lens = [20, 18, 2, 1], [36, 18, 1, 30]
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = c.clone()
    vdx.rope3d_append(x, x, x, c.cache(vdx), cu_of(news), kv_len, (29, 1, 1))
    with pytest.raises(vdx.VdxError):
        vdx.sync_check()
    vdx.sync_check()
    changed = (c.v.view(torch.uint8) != before.v.view(torch.uint8)).flatten(2).any(-1)
    want = torch.zeros_like(changed)
    want[1, :13] = True            # sequence 0: indices 16 .. 31, of which the grid has 28
    want[2, :2] = True             # sequence 1: its second page
    want[3, 0] = True              # sequence 2: index 0 (the row before it has index -1)
    assert torch.equal(changed, want), changed.nonzero()
    sc = (c.v_scale.view(torch.uint8) != before.v_scale.view(torch.uint8)).flatten(1).any(-1)
    assert sc.tolist() == [i in (1, 2, 3) for i in range(sc.shape[0])]


# ------------------------------------------------------------------------------------------------ attention
PAGED = [
    # dtype, d, Hq, Hkv, page, new tokens, keys, block
    ("bf16", 128, 12, 12, 16, [1] * 5, [1, 15, 17, 300, 1000], 0),
    ("bf16", 128, 40, 8, 64, [1, 1, 1], [3000, 1, 777], 1),
    ("fp16", 64, 12, 4, 16, [1, 3, 2], [700, 33, 2], 1),
    ("fp16", 128, 8, 1, 200, [2, 1], [999, 200], 0),
    ("bf16", 64, 4, 4, 129, [7, 8, 1], [515, 8, 130], 3),
    ("bf16", 128, 2, 1, 32, [9, 0, 16], [600, 50, 16], 4),
    ("bf16", 128, 1, 1, 128, [1], [40000], 0),
    ("fp16", 64, 16, 1, 64, [1, 2], [20000, 5000], 1),
    ("bf16", 128, 4, 4, 16, [40, 33, 1], [500, 33, 70], 1),
    ("fp16", 64, 12, 4, 32, [129, 300, 64], [129, 1200, 700], 16),
    ("bf16", 128, 3, 3, 1560, [260, 100], [2000, 1661], 0),
    ("fp16", 128, 12, 1, 200, [50, 77], [801, 199], 7),
    ("bf16", 64, 5, 1, 129, [300], [901], 0),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"{c[0]}-d{c[1]}-{c[2]}over{c[3]}-page{c[4]}-{max(c[5])}of{max(c[6])}-block{c[7]}")
@pytest.mark.parametrize("order", ["token", "head"])
def test_attention_over_8_bits_matches_the_formula(case, order):
    dtype, d, Hq, Hkv, page, news, lens, block = case
    dt = DT[dtype]
    c = Paged8(d, Hkv, page, lens, seed=21, order=order, scale_order="page" if order == "head" else "head")
    q = _rand((sum(news) + 2, Hq, d), dt, 22, 0.7)
    out, lse = vdx.paged_attn(q, c.cache(vdx), cu_of(news), c.kv_len, max_q=max(news), max_kv=max(lens), causal_block=block)
    vdx.sync_check()
    at = 0
    for s, n in enumerate(news):
        ref = attend(q[at:at + n], c.get(c.k, c.k_scale, s), c.get(c.v, c.v_scale, s), limits(n, lens[s], block))
        check_attention8(out[at:at + n], lse[:, at:at + n], ref, dt, f"sequence {s}")
        at += n


@pytest.mark.parametrize("n", [1, 40])
def test_rows_that_see_nothing_and_rows_of_no_sequence(n):
    d, H, dt = 128, 2, torch.bfloat16
    c = Paged8(d, H, 16, [0, 30], seed=5, width=4)
    q = _rand((2 * n + 4, H, d), dt, 6)
    out, lse = torch.full_like(q, 7.0), torch.full((H, 2 * n + 4), 7.0, device="cuda")
    vdx.paged_attn(q, c.cache(vdx), cu_of([n, n]), c.kv_len, max_q=n, out=out, lse=lse)
    vdx.sync_check()
    assert bool((out[:n] == 0).all()) and bool((lse[:, :n] == -math.inf).all())
    assert bool((out[2 * n:] == 7).all()) and bool((lse[:, 2 * n:] == 7).all())
    ref = attend(q[n:2 * n], c.get(c.k, c.k_scale, 1), c.get(c.v, c.v_scale, 1), limits(n, 30, 0))
    check_attention8(out[n:2 * n], lse[:, n:2 * n], ref, dt)


@pytest.mark.parametrize("n", [1, 50])
@pytest.mark.parametrize("gain", [2.0 ** -100, 2.0 ** -20, 1.0, 300.0, 2.0 ** 40])
def test_queries_of_any_size(n, gain):
    # queries of bf16 are brought into fp16's range: nothing may over- or underflow on the way
    d, H, dt = 128, 2, torch.bfloat16
    c = Paged8(d, H, 64, [200], seed=7)
    q = _rand((n, H, d), dt, 8, gain)
    q[:, 1, 64:] *= 2.0 ** -12
    scale = 0.3 / gain
    out, lse = vdx.paged_attn(q, c.cache(vdx), cu_of([n]), c.kv_len, scale=scale)
    vdx.sync_check()
    scale = float(torch.tensor(scale, dtype=torch.float32))
    ref = attend(q, c.get(c.k, c.k_scale, 0), c.get(c.v, c.v_scale, 0), limits(n, 200, 0), scale)
    check_attention8(out, lse, ref, dt)


@pytest.mark.parametrize("n", [1, 40])
def test_8_bit_pages_and_lengths_out_of_range_are_reported(n):
    d, H, dt = 64, 2, torch.bfloat16
    c = Paged8(d, H, 16, [40, 40], seed=9)
    q, cu = _rand((2 * n, H, d), dt, 10), cu_of([n, n])
    table = c.table.clone()
    c.table[0, 1] = c.k.shape[0]
    out, lse = vdx.paged_attn(q, c.cache(vdx), cu, c.kv_len, max_q=n)
    with pytest.raises(vdx.VdxError, match="page"):
        vdx.sync_check()
    k, v = (x.clone() for x in (c.get(c.k, c.k_scale, 1), c.get(c.v, c.v_scale, 1)))
    check_attention8(out[n:], lse[:, n:], attend(q[n:], k, v, limits(n, 40, 0)), dt)
    c.table.copy_(table)
    k, v = c.get(c.k, c.k_scale, 0), c.get(c.v, c.v_scale, 0)
    k[16:32] = 0
    v[16:32] = 0
    check_attention8(out[:n], lse[:, :n], attend(q[:n], k, v, limits(n, 40, 0)), dt)
    vdx.paged_attn(q, c.cache(vdx), cu, c.kv_len + 100, max_q=n)
    with pytest.raises(vdx.VdxError, match="kv_len"):
        vdx.sync_check()


def test_what_is_refused_of_8_bit_caches():
    d, H, dt = 128, 2, torch.bfloat16
    c = Paged8(d, H, 16, [40, 9], seed=70)
    x, cu = _rand((2, H, d), dt, 71), cu_of([1, 1])
    good = c.cache(vdx)
    P = vdx.PagedKV
    bad = [
        P(c.k, c.v, c.table), P(c.k, c.v, c.table, c.k_scale, None), P(c.k, c.v, c.table, c.k_scale, c.v_scale[:1]),
        P(c.k, c.v, c.table, c.k_scale.view(torch.uint8), c.v_scale), P(c.k, c.v.view(torch.uint8), c.table, c.k_scale, c.v_scale),
        P(c.k.view(torch.uint8), c.v.view(torch.uint8), c.table, c.k_scale, c.v_scale),
        P(c.k, c.v, c.table, c.k_scale.cpu(), c.v_scale), P(c.k, c.v, c.table, c.k_scale[:, :, :1], c.v_scale[:, :, :1]),
        P(c.k.float().to(dt), c.v.float().to(dt), c.table, c.k_scale, c.v_scale),
    ]
    for i, cache in enumerate(bad):
        for f in (lambda: vdx.paged_attn(x, cache, cu, c.kv_len), lambda: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (99, 1, 1)),
                  lambda: vdx.paged_attn_workspace_bytes(x, cache, cu, c.kv_len)):
            with pytest.raises(vdx.VdxError):
                f()
                pytest.fail(f"cache {i} was taken")
    for f in (lambda: vdx.paged_attn(x.float(), good, cu, c.kv_len), lambda: vdx.paged_attn(x.view(torch.uint8)[..., :d].view(CODE), good, cu, c.kv_len),
              lambda: vdx.rope3d_append(x, x, x.half(), good, cu, c.kv_len, (99, 1, 1)),
              lambda: vdx.rope3d_append(x, x.cpu(), x.cpu(), good, cu, c.kv_len, (99, 1, 1)),
              lambda: vdx.rope3d_append(x, x, x, P(c.k, c.v, c.table, c.k_scale, c.k_scale), cu, c.kv_len, (99, 1, 1)),
              lambda: vdx.rope3d_append(x, x, x, P(c.k, c.k, c.table, c.k_scale, c.v_scale), cu, c.kv_len, (99, 1, 1)),
              lambda: vdx.paged_attn(x.clone().requires_grad_(), good, cu, c.kv_len)):
        with pytest.raises(vdx.VdxError):
            f()
    versions = [t._version for t in (c.k, c.v, c.k_scale, c.v_scale)]
    vdx.rope3d_append(x, x, x, good, cu, c.kv_len, (99, 1, 1))
    assert [t._version for t in (c.k, c.v, c.k_scale, c.v_scale)] == [n + 1 for n in versions]
    vdx.sync_check()


assert SCALE
