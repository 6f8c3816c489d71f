"""Gathered attention weights and eviction, over caches of 16 and 8 bits, against the definition."""
import math

import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from kv8_ref import BLOCK, Paged8, stay, weigh
from streaming_ref import DT, Paged, attend, cu_of, limits

pytestmark = pytest.mark.gpu


def _rand(shape, dtype, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def _cache(bits, dt, d, Hkv, page, lens, seed, **kw):
    """A cache and its keys and values by sequence, in 64 bits."""
    if bits == 8:
        c = Paged8(d, Hkv, page, lens, seed, **kw)
        return c, c.cache(vdx), lambda s: (c.get(c.k, c.k_scale, s), c.get(c.v, c.v_scale, s))
    c = Paged(dt, d, Hkv, page, lens, seed, **kw)
    return c, vdx.PagedKV(c.k, c.v, c.table), lambda s: tuple(x.double() for x in c.get(s))


# ------------------------------------------------------------------------------------------------ gathered weights
WEIGH = [
    # dtype, d, Hq, Hkv, page, new tokens, keys, block, decay
    ("bf16", 128, 12, 12, 16, [1] * 5, [1, 15, 17, 300, 1000], 0, 1.0),
    ("bf16", 128, 40, 8, 64, [1, 1, 1], [3000, 1, 777], 1, 0.9),
    ("fp16", 64, 12, 4, 16, [1, 3, 2], [700, 33, 2], 1, 1.0),
    ("fp16", 128, 8, 1, 200, [2, 0, 1], [999, 50, 200], 0, 0.5),
    ("bf16", 64, 4, 4, 129, [7, 8, 1], [515, 8, 130], 3, 1.0),
    ("bf16", 128, 2, 1, 32, [9, 0, 16], [600, 50, 16], 4, 0.0),
    ("bf16", 128, 4, 4, 16, [40, 33, 1], [500, 33, 70], 1, 1.0),
    ("fp16", 64, 12, 4, 32, [129, 300, 64], [129, 1200, 700], 16, -0.5),
    ("bf16", 128, 3, 3, 1560, [260, 100], [2000, 1661], 0, 1.0),
    ("fp16", 128, 12, 1, 200, [50, 77], [801, 199], 7, 0.9),
    ("bf16", 64, 5, 1, 129, [300], [901], 0, 1.0),
    ("bf16", 128, 8, 2, 128, [513, 130], [2600, 130], 100, 1.0),
]


# more units of 256 keys than multiprocessors, of no, few and many query tiles one after another in a block
WEIGH += [
    ("bf16", 128, 8, 8, 64, [600, 40, 0, 1200, 130, 33], [1500, 1490, 700, 1290, 1025, 1501], 1, 1.0),
    ("fp16", 64, 12, 6, 16, [33, 700, 40, 1, 90, 1030], [1280, 1100, 1, 257, 1800, 1030], 50, 0.75),
]


@pytest.mark.parametrize("case", WEIGH, ids=lambda c: f"{c[0]}-d{c[1]}-{c[2]}over{c[3]}-page{c[4]}-{max(c[5])}of{max(c[6])}-block{c[7]}")
@pytest.mark.parametrize("bits", [16, 8])
def test_gathered_weights_match_the_formula(case, bits):
    dtype, d, Hq, Hkv, page, news, lens, block, decay = case
    dt = DT[dtype]
    c, cache, values = _cache(bits, dt, d, Hkv, page, lens, 31, order="head" if d == 64 else "token")
    rows, width = sum(news), max(lens) + 5
    q = _rand((rows, Hq, d), dt, 32, 0.7)
    _, lse = vdx.paged_attn(q, cache, cu_of(news), c.kv_len, max_q=max(news), max_kv=max(lens), causal_block=block)
    pool = _rand((len(lens), Hkv + 1, width + 3), torch.float32, 33).abs()
    w = pool[:, :Hkv, 1:1 + width]
    before = pool.clone()
    assert vdx.paged_attn_weights(q, cache, cu_of(news), c.kv_len, lse, w, max_q=max(news), max_kv=max(lens), causal_block=block,
                                  decay=decay) is w
    vdx.sync_check()
    want, at = before.double(), 0
    bound = torch.zeros_like(want)
    for s, n in enumerate(news):
        L = lens[s]
        if n:
            mine = want[s, :Hkv, 1:1 + L]
            mine[:, :max(0, L - n)] *= float(torch.tensor(decay, dtype=torch.float32))
            mine[:, max(0, L - n):] = 0
            bound[s, :Hkv, 1:1 + L] = 2.0 ** -22 * mine.abs()
            add, b = weigh(q[at:at + n], values(s)[0], limits(n, L, block), lse[:, at:at + n])
            mine += add
            bound[s, :Hkv, 1:1 + L] += b + 2.0 ** -22 * mine.abs()
        at += n
    err = (pool.double() - want).abs()
    assert bool((err <= bound).all()), (float((err / bound.clamp_min(1e-300)).max()), float(err.max()))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [2, 150])
def test_weights_of_a_sequence_sum_to_its_rows(bits, n):
    c, cache, _ = _cache(bits, torch.bfloat16, 128, 2, 64, [900], 41)
    w, total = torch.full((1, 2, 900), math.nan, device="cuda"), 0
    for end in (n, 400, 900):
        q = _rand((n, 6, 128), torch.bfloat16, 42 + end)
        kv_len = torch.tensor([end], dtype=torch.int32, device="cuda")
        _, lse = vdx.paged_attn(q, cache, cu_of([n]), kv_len, causal_block=1)
        if end > n:                              # keys between the calls: appended without attention
            w[:, :, total:end - n] = 0
        vdx.paged_attn_weights(q, cache, cu_of([n]), kv_len, lse, w, causal_block=1)
        total = end
    vdx.sync_check()
    assert bool(((w.double().sum(-1) - 3 * 3 * n).abs() < 1e-3 * n).all())


@pytest.mark.parametrize("n", [3, 70])
def test_rows_without_keys_and_nan_rows(n):
    d, dt = 64, torch.bfloat16
    c, cache, values = _cache(16, dt, d, 2, 16, [n + 20, 40], 51)
    q = _rand((2 * n, 2, d), dt, 52)
    _, lse = vdx.paged_attn(q, cache, cu_of([n, n]), c.kv_len, causal_block=1)
    lse[:, 0] = -math.inf                        # a row that is told to have seen nothing
    lse[1, n] = math.nan                         # head 1 of sequence 1's first row
    w = torch.zeros(2, 2, 200, device="cuda")
    vdx.paged_attn_weights(q, cache, cu_of([n, n]), c.kv_len, lse, w, causal_block=1)
    vdx.sync_check()
    add, b = weigh(q[:n], values(0)[0], limits(n, n + 20, 1), lse[:, :n])
    assert bool(((w[0, :, :n + 20].double() - add).abs() <= b + 2.0 ** -22 * add).all())
    seen = int(limits(n, 40, 1)[0])
    assert bool(torch.isnan(w[1, 1, :seen]).all()) and not bool(torch.isnan(w[1, 1, seen:]).any()) and not bool(torch.isnan(w[1, 0]).any())


def test_weights_report_lengths_and_pages_and_refuse_what_they_cannot_take():
    d, dt = 128, torch.bfloat16
    c, cache, _ = _cache(16, dt, d, 2, 16, [40, 30], 61)
    q, cu = _rand((2, 4, d), dt, 62), cu_of([1, 1])
    _, lse = vdx.paged_attn(q, cache, cu, c.kv_len)
    w = torch.zeros(2, 2, 35, device="cuda")
    vdx.paged_attn_weights(q, cache, cu, c.kv_len, lse, w)             # 40 keys, 35 places
    with pytest.raises(vdx.VdxError, match="kv_len"):
        vdx.sync_check()
    c.table[1, 0] = -1
    vdx.paged_attn_weights(q, cache, cu, c.kv_len, lse, torch.zeros(2, 2, 48, device="cuda"))
    with pytest.raises(vdx.VdxError, match="page"):
        vdx.sync_check()
    args = (q, cache, cu, c.kv_len)
    for bad in (lambda: vdx.paged_attn_weights(*args, lse[:1], w), lambda: vdx.paged_attn_weights(*args, lse, w.double()),
                lambda: vdx.paged_attn_weights(*args, lse, w[0]), lambda: vdx.paged_attn_weights(*args, lse, w.transpose(0, 2)),
                lambda: vdx.paged_attn_weights(*args, lse, w[:, :1]), lambda: vdx.paged_attn_weights(*args, lse, w[:1].expand(2, 2, 35)),
                lambda: vdx.paged_attn_weights(*args, lse, w, decay=math.nan), lambda: vdx.paged_attn_weights(*args, lse.cpu(), w),
                lambda: vdx.paged_attn_weights(*args, lse, lse.view(2, 2, 2)[:, :, :2]), lambda: vdx.paged_attn_weights(*args, None, w),
                lambda: vdx.paged_attn_weights(*args, lse, w.clone().requires_grad_())):
        with pytest.raises(vdx.VdxError):
            bad()
    version = w._version
    vdx.paged_attn_weights(*args[:3], c.kv_len.clamp(max=35), lse, w)
    assert w._version == version + 1
    with pytest.raises(vdx.VdxError):
        vdx.sync_check()


# ------------------------------------------------------------------------------------------------ eviction
def _into(bits, dt, d, Hkv, page, lens, keep, seed, **kw):
    kept = [min(n, keep) for n in lens]
    c, cache, values = _cache(bits, dt, d, Hkv, page, [0] * len(lens), seed, spare=sum(-(-n // page) for n in kept) + 2,
                              width=max(1, max(-(-n // page) for n in kept)), **kw)
    perm = torch.randperm(c.k.shape[0], generator=torch.Generator().manual_seed(seed)).tolist()
    for s, n in enumerate(kept):
        for i in range(-(-n // page)):
            c.table[s, i] = perm.pop()
    c.lens = kept
    return c, cache, values


def _check_evicted(got, into, before, c, weights, lens, keep, recent, bits, offset):
    """into: the new cache after the call, before: as it was; c: the old cache, as it was."""
    assert got.kv_len.tolist() == [min(n, keep) for n in lens]
    assert got.pos_offset.tolist() == [o + n - min(n, keep) for o, n in zip(offset, lens)]
    if bits == 8:
        want = before.clone()
    else:
        want = Paged.__new__(Paged)
        want.__dict__.update(before.__dict__)
        want.k, want.v = before.k.clone(), before.v.clone()
    for s, L in enumerate(lens):
        left = min(L, keep)
        kept = [stay(weights[s, h], L, keep, recent) for h in range(c.Hkv)]
        for h in range(c.Hkv):
            assert got.index[s, h].tolist() == kept[h] + [-1] * (keep - left), (s, h)
            w = got.weights[s, h, :keep]
            assert torch.equal(w[:left].nan_to_num(9e9), weights[s, h][kept[h]].nan_to_num(9e9)) and bool((w[left:] == 0).all())
        if left == 0:
            continue
        idx = torch.tensor(kept, device="cuda").T                       # [left, Hkv]
        heads = torch.arange(c.Hkv, device="cuda")[None]
        if bits == 8:
            for codes, scales, wc, ws in ((c.k, c.k_scale, want.k, want.k_scale), (c.v, c.v_scale, want.v, want.v_scale)):
                want.put(wc, ws, s, 0, c.get(codes, scales, s, L)[idx, heads])
        else:
            page, slot = want.slots(s, torch.arange(left, device="cuda"))
            k, v = c.get(s, L)
            want.k[page, slot], want.v[page, slot] = k[idx, heads], v[idx, heads]
    def raw(t):
        return t.contiguous().view(torch.uint8)
    for n in ("k", "v") + (("k_scale", "v_scale") if bits == 8 else ()):
        assert torch.equal(raw(getattr(into, n)), raw(getattr(want, n))), n


EVICT = [
    # dtype, d, Hkv, page, page of the new table, keys, keep, recent
    ("bf16", 128, 3, 16, 16, [300, 50, 17, 0, 16], 50, 7),
    ("fp16", 64, 2, 32, 16, [100, 33, 5000], 33, 33),
    ("bf16", 64, 5, 200, 129, [999, 450, 130], 450, 0),
    ("bf16", 128, 1, 64, 200, [20000, 1], 7777, 1000),
    ("fp16", 128, 2, 129, 64, [257, 130], 1, 0),
    ("bf16", 128, 2, 128, 128, [4096, 4097, 4095], 4096, 4095),
    ("bf16", 64, 1, 16, 32, [9], 400, 3),
]


@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{c[0]}-d{c[1]}-{c[2]}heads-page{c[3]}to{c[4]}-{max(c[5])}to{c[6]}")
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_eviction_matches_the_definition(case, bits, kind):
    dtype, d, Hkv, page, page_to, lens, keep, recent = case
    dt = DT[dtype]
    c, cache, _ = _cache(bits, dt, d, Hkv, page, lens, 81, order="head" if d == 64 else "token")
    into, into_cache, _ = _into(bits, dt, d, Hkv, page_to, lens, keep, 82)
    if bits == 8:
        before = into.clone()
    else:
        before = Paged.__new__(Paged)
        before.__dict__.update(into.__dict__)
        before.k, before.v = into.k.clone(), into.v.clone()
    w = torch.exp(3 * _rand((len(lens), Hkv, max(lens) + 2), torch.float32, 83))
    if kind == "ties":
        g = torch.Generator(device="cuda").manual_seed(84)
        w = torch.randint(0, 4, w.shape, generator=g, device="cuda").float() - 1
        w[w == 0] = torch.where(torch.rand(int((w == 0).sum()), generator=g, device="cuda") < 0.5, 0.0, -0.0)
        pick = torch.rand(w.shape, generator=g, device="cuda")
        w[pick < 0.02] = math.inf
        w[(pick > 0.02) & (pick < 0.03)] = -math.inf
        w[(pick > 0.03) & (pick < 0.04)] = math.nan
    kept_w, offset = w.clone(), [5 * s - 3 for s in range(len(lens))]
    got = vdx.paged_evict(cache, w, c.kv_len, keep, into_cache, recent=recent, max_kv=max(lens),
                          pos_offset=torch.tensor(offset, dtype=torch.int32, device="cuda"))
    vdx.sync_check()
    assert torch.equal(w.view(torch.int32), kept_w.view(torch.int32))
    _check_evicted(got, into, before, c, kept_w, lens, keep, recent, bits, offset)


@pytest.mark.parametrize("L", [120, 9000])
@pytest.mark.parametrize("keep", [30, 31, 60, 90])
def test_borders_between_groups_of_alike_weights(L, keep):
    # quarters of the keys far apart, near each other and the least that there are: where the border falls between groups that
    # share their upper bits, inside one, and among equals
    d, H, dt = 64, 3, torch.bfloat16
    c, cache, _ = _cache(16, dt, d, H, 64, [L], 91)
    keep = keep * L // 120
    into, into_cache, _ = _into(16, dt, d, H, 64, [L], keep, 92)
    before = Paged.__new__(Paged)
    before.__dict__.update(into.__dict__)
    before.k, before.v = into.k.clone(), into.v.clone()
    group = torch.randperm(L, generator=torch.Generator().manual_seed(93)).cuda() % 4
    rest = torch.rand(1, H, L, generator=torch.Generator(device="cuda").manual_seed(94), device="cuda")
    w = torch.empty(1, H, L, device="cuda")
    w[:, 0] = torch.tensor([-math.inf, 2.0 ** -60, 1.0, 2.0 ** 60], device="cuda")[group] * (1 + 0.9 * rest[:, 0])
    w[:, 1] = 1 + group * 2.0 ** -7 + rest[:, 1] * 2.0 ** -9
    w[:, 2] = torch.tensor([-math.inf, -math.inf, -0.0, 5.0], device="cuda")[group]
    got = vdx.paged_evict(cache, w, c.kv_len, keep, into_cache)
    vdx.sync_check()
    _check_evicted(got, into, before, c, w, [L], keep, 0, 16, [0])


def test_eviction_in_one_pool_with_weights_in_place_and_on_a_side_stream():
    bits, dt, d, H, page, lens, keep = 8, torch.bfloat16, 128, 2, 16, [5000, 300, 60], 130
    c = Paged8(d, H, page, lens, seed=91, spare=30, width=320)
    used = set(c.table[c.table >= 0].tolist())
    free = [i for i in range(c.k.shape[0]) if i not in used]
    table = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(lens):
        for i in range(-(-min(n, keep) // page)):
            table[s, i] = free.pop()
    before = c.clone()
    w = torch.exp(_rand((3, H, 5100), torch.float32, 92))
    first = w.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    into = vdx.PagedKV(c.k, c.v, table, c.k_scale, c.v_scale)
    got = vdx.paged_evict(c.cache(vdx), w, c.kv_len, keep, into, recent=9, weights_out=w, stream=side)
    side.synchronize()
    vdx.sync_check()
    assert got.weights is w and torch.equal(w[:, :, keep:], first[:, :, keep:])
    after, start = c.clone(), before.clone()
    after.table = start.table = table
    _check_evicted(got, after, start, before, first, lens, keep, 9, bits, [0, 0, 0])


def test_what_eviction_refuses_and_reports():
    dt, d, H = torch.bfloat16, 64, 2
    c, cache, _ = _cache(16, dt, d, H, 16, [40, 30], 95)
    into, to, _ = _into(16, dt, d, H, 16, [40, 30], 20, 96)
    w = torch.rand(2, H, 48, device="cuda")
    eight, eight_cache, _ = _cache(8, dt, d, H, 16, [40, 30], 97)
    other, other_cache, _ = _cache(16, dt, d, H + 1, 16, [40, 30], 98)
    three, three_cache, _ = _cache(16, dt, d, H, 16, [40, 30, 1], 98)
    half, half_cache, _ = _cache(16, torch.float16, d, H, 16, [40, 30], 99)
    E = vdx.paged_evict
    for bad in (lambda: E(cache, w, c.kv_len, 0, to), lambda: E(cache, w, c.kv_len, 5, to, recent=6), lambda: E(cache, w, c.kv_len, 5, cache),
                lambda: E(cache, w, c.kv_len, 5, eight_cache), lambda: E(cache, w, c.kv_len, 5, other_cache), lambda: E(cache, w, c.kv_len, 5, three_cache),
                lambda: E(cache, w, c.kv_len, 5, half_cache), lambda: E(cache, w.double(), c.kv_len, 5, to), lambda: E(cache, w[:1], c.kv_len, 5, to),
                lambda: E(cache, w, c.kv_len.long(), 5, to), lambda: E(cache, w, c.kv_len, 5, to, weights_out=w[:, :, :4]),
                lambda: E(cache, w, c.kv_len, 5, to, weights_out=w[:, :, 1:]), lambda: E(cache, w, c.kv_len, 5, to, recent=-1),
                lambda: E(cache, w, c.kv_len, 5, vdx.PagedKV(c.k, into.v, into.table)),
                lambda: E(cache, w, c.kv_len, 5, vdx.PagedKV(c.k[1:], c.v[1:], into.table)),
                lambda: E(cache, w, c.kv_len, 5, vdx.PagedKV(into.k, into.k, into.table)),
                lambda: E(cache, w.clone().requires_grad_(), c.kv_len, 5, to), lambda: E(cache, w, None, 5, to)):
        with pytest.raises(vdx.VdxError):
            bad()
    vdx.sync_check()
    E(cache, w, torch.tensor([50, 30], dtype=torch.int32, device="cuda"), 20, to)      # 50 keys in a table of 48
    with pytest.raises(vdx.VdxError, match="kv_len"):
        vdx.sync_check()
    small = vdx.PagedKV(into.k, into.v, into.table[:, :1].contiguous())
    before = into.k.clone()
    got = E(cache, w, c.kv_len, 20, small)                  # a table that holds 16 of 20
    with pytest.raises(vdx.VdxError, match="page table"):
        vdx.sync_check()
    rest = torch.ones(into.k.shape[0], dtype=torch.bool, device="cuda")
    rest[into.table[:, 0].long()] = False
    assert torch.equal(into.k[rest].view(torch.int16), before[rest].view(torch.int16)) and got.kv_len.tolist() == [20, 20]
    c.table[0, 2] = 77
    E(cache, torch.ones_like(w), c.kv_len, 20, to, recent=20)
    with pytest.raises(vdx.VdxError, match="page index"):
        vdx.sync_check()
    k = into.k[into.table[0].long()].flatten(0, 1)[:20]
    assert bool((k[12:] == 0).all()) and not bool((k[:12] == 0).all(-1).any())      # keys 20 .. 39; those of the third page
    vdx.sync_check()


assert attend and BLOCK
