"""Appending, attention, gathered weights and eviction together, as a generation that is kept short runs them: over
caches of 16 and 8 bits, in bare chains, in graphs, on streams, and where offsets are large."""
import math

import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from kv8_ref import BLOCK, CODE, SCALE, Paged8, check_attention8, codes64, half_step8, least_exponent, powers, stay, weigh
from streaming_ref import SECTIONS, attend, check_attention, cu_of, half_step, limits, rotate, rotate_bound

pytestmark = pytest.mark.gpu


def _rand(shape, dtype, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


class Pool:
    """Keys and values of 16 or 8 bits, and page tables over them."""

    def __init__(self, bits, dt, d, H, page, pages):
        self.bits, self.page, self.free = bits, page, list(range(pages))
        shape = (pages, page, H, d)
        if bits == 8:
            self.k, self.v = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(CODE) for _ in range(2))
            self.ks, self.vs = (torch.full((pages, -(-page // BLOCK), H), 0xff, dtype=torch.uint8, device="cuda").view(SCALE) for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=dt, device="cuda") for _ in range(2))
            self.ks = self.vs = None

    def cache(self, table):
        return vdx.PagedKV(self.k, self.v, table, self.ks, self.vs)

    def values(self, table, s, n, which):
        """[n, H, d] of sequence s in 64 bits."""
        c = torch.arange(n, device="cuda")
        pg, sl = table[s].long()[c // self.page], c % self.page
        x = self.k if which == "k" else self.v
        if self.bits == 16:
            return x[pg, sl].double()
        sc = self.ks if which == "k" else self.vs
        return codes64(x.view(torch.uint8)[pg, sl]) * powers(sc.view(torch.uint8)[pg, sl // BLOCK].int() - 127)[..., None]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dt,d,Hq,Hkv,page,chunk,block,keep,recent", [
    (torch.bfloat16, 128, 4, 2, 16, 1, 1, 40, 8),
    (torch.float16, 64, 6, 2, 32, 24, 24, 130, 48),
    (torch.bfloat16, 128, 2, 2, 200, 90, 30, 300, 0),
])
def test_a_generation_that_is_kept_short(bits, dt, d, Hq, Hkv, page, chunk, block, keep, recent):
    # each step appends a chunk to two sequences, attends, adds up the weights and, past a length, evicts into fresh pages
    S, steps = 2, 14
    most = keep + 4 * chunk + 30
    width = -(-most // page)
    pool = Pool(bits, dt, d, Hkv, page, 6 * width + 4)
    grid = (4000, 1, 1)
    table = torch.zeros((S, width), dtype=torch.int32, device="cuda")
    for s in range(S):
        for i in range(width):
            table[s, i] = pool.free.pop()
    lens, offs = [0, 0], [0, 0]
    w = torch.full((S, Hkv, most), math.nan, device="cuda")
    want_w = [torch.zeros(Hkv, 0, dtype=torch.float64, device="cuda") for _ in range(S)]
    bound_w = [torch.zeros_like(x) for x in want_w]
    evicted = 0
    for step in range(steps):
        n = chunk if step else keep - chunk                                # the first chunk is long
        lens = [x + n for x in lens]
        kv_len, off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, offs))
        x = _rand((S * n, Hq + 2 * Hkv, d), dt, 200 + step, 1.2)
        cache, cu = pool.cache(table), cu_of([n] * S)
        q = vdx.rope3d_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, cu, kv_len, grid, SECTIONS[d], pos_offset=off)
        out, lse = vdx.paged_attn(q, cache, cu, kv_len, max_q=n, max_kv=most, causal_block=block, pos_offset=off)
        vdx.paged_attn_weights(q, cache, cu, kv_len, lse, w, max_q=n, max_kv=most, causal_block=block, pos_offset=off, decay=0.9)
        vdx.sync_check()
        decay = float(torch.tensor(0.9, dtype=torch.float32))
        for s in range(S):
            L = lens[s]
            pos = torch.arange(L - n, L, device="cuda") + offs[s]
            rows = slice(s * n, (s + 1) * n)
            ref_q = rotate(x[rows, :Hq], pos, grid, SECTIONS[d], 10000.0)
            assert bool(((q[rows].double() - ref_q).abs() <= rotate_bound(ref_q, dt)).all())
            k, v = pool.values(table, s, L, "k"), pool.values(table, s, L, "v")
            ref_k = rotate(x[rows, Hq:Hq + Hkv], pos, grid, SECTIONS[d], 10000.0)
            if bits == 16:
                assert bool(((k[-n:] - ref_k).abs() <= rotate_bound(ref_k, dt)).all())
            else:                                                          # half a step of the largest scale that the chunk can have
                unit = powers(least_exponent(k.abs().amax((0, 2)) * 1.01))[None, :, None]
                assert bool(((k[-n:] - ref_k).abs() <= half_step8(ref_k / unit) * unit * 1.01 + 2.0 ** -18 * ref_k.abs().amax()).all())
            # blocks are counted from grid token 0
            p = pos
            limit = (((p // block) + 1) * block - offs[s]).clamp(max=L)
            ref = attend(q[rows], k, v, limit)
            (check_attention if bits == 16 else check_attention8)(out[rows], lse[:, rows], ref, dt, f"step {step}")
            add, b = weigh(q[rows], k, limit, lse[:, rows])
            old = torch.nn.functional.pad(want_w[s] * decay, (0, n))
            want_w[s] = old + add
            bound_w[s] = torch.nn.functional.pad(bound_w[s] * decay, (0, n)) + b + 2.0 ** -22 * want_w[s]
            assert bool(((w[s, :, :L].double() - want_w[s]).abs() <= bound_w[s]).all())
        if max(lens) <= keep + 2 * chunk:
            continue
        evicted += 1
        fresh = torch.zeros_like(table)
        for s in range(S):
            for i in range(width):
                fresh[s, i] = pool.free.pop()
        before = [[pool.values(table, s, lens[s], a) for a in "kv"] for s in range(S)]
        kept_w = w.clone()
        left = vdx.paged_evict(cache, w, kv_len, keep, pool.cache(fresh), recent=recent, max_kv=most, pos_offset=off, weights_out=w)
        vdx.sync_check()
        pool.free += table.flatten().tolist()                              # the old pages are free
        table = fresh
        assert left.kv_len.tolist() == [min(x, keep) for x in lens]
        for s in range(S):
            kept = [stay(kept_w[s, h], lens[s], keep, recent) for h in range(Hkv)]
            assert left.index[s].tolist() == [x + [-1] * (keep - len(x)) for x in kept]
            idx, heads = torch.tensor(kept, device="cuda").T, torch.arange(Hkv, device="cuda")[None]
            for a, full in zip("kv", before[s]):
                got, want = pool.values(table, s, idx.shape[0], a), full[idx, heads]
                if bits == 16:
                    assert torch.equal(got, want)
                else:                                                      # exact, but for what becomes subnormal
                    assert bool(((got - want).abs() <= 2.0 ** -10 * powers(least_exponent(want.abs().amax((0, 2))))[None, :, None]).all())
            want_w[s], bound_w[s] = want_w[s][heads.T, idx.T], bound_w[s][heads.T, idx.T]
        offs = left.pos_offset.tolist()
        lens = left.kv_len.tolist()
    assert evicted >= 2 and offs[0] > 0 and half_step(dt) > 0


def _state(bits, seed, n, S=3, H=4, d=128, page=16, ctx=200):
    dt = torch.bfloat16
    lens = [ctx + 37 * s + n for s in range(S)]
    width = -(-max(lens) // page) + 1
    pool = Pool(bits, dt, d, H, page, 2 * S * width)
    order = torch.randperm(2 * S * width, generator=torch.Generator().manual_seed(seed)).int().cuda()
    tables = order[:S * width].view(S, width).clone(), order[S * width:].view(S, width).clone()
    first = _rand((sum(lens), 2, H, d), dt, seed)
    vdx.rope3d_append(None, first[:, 0], first[:, 1], pool.cache(tables[0]), cu_of(lens), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      (9999, 1, 1))
    w = _rand((S, H, width * page), torch.float32, seed + 1).abs()
    x = _rand((S * n, 3 * H, d), dt, seed + 2)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    off = torch.zeros(S, dtype=torch.int32, device="cuda")
    return dict(pool=pool, tables=tables, w=w, x=x, kv_len=kv_len, off=off, cu=cu_of([n] * S), n=n, H=H, top=width * page)


def _step(st, keep=100, sync=False):
    pool, H, n = st["pool"], st["H"], st["n"]
    cache, into = pool.cache(st["tables"][0]), pool.cache(st["tables"][1])
    x, cu, kv_len = st["x"], st["cu"], st["kv_len"]
    wait = torch.cuda.synchronize if sync else lambda: None
    q = vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], cache, cu, kv_len, (9999, 1, 1), pos_offset=st["off"])
    wait()
    out, lse = vdx.paged_attn(q, cache, cu, kv_len, max_q=n, max_kv=st["top"], causal_block=1)
    wait()
    vdx.paged_attn_weights(q, cache, cu, kv_len, lse, st["w"], max_q=n, max_kv=st["top"], causal_block=1)
    wait()
    left = vdx.paged_evict(cache, st["w"], kv_len, keep, into, recent=20, pos_offset=st["off"])
    wait()
    return [q, out, lse, st["w"].clone(), *left] + [t.view(torch.uint8).clone() for t in (pool.k, pool.v, pool.ks, pool.vs) if t is not None]


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [1, 50])
def test_bare_chains_and_side_streams_give_the_same_bits(bits, n):
    want = _step(_state(bits, 7, n), sync=True)
    for trial in range(3):
        st = _state(bits, 7, n)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side if trial else torch.cuda.current_stream()):
            got = _step(st)
        torch.cuda.synchronize()
        assert _same(got, want), trial
    vdx.sync_check()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [1, 70])
def test_a_captured_step_replays_with_new_lengths_and_inputs(bits, n):
    st = _state(bits, 9, n)
    start = [t.view(torch.uint8).clone() for t in (st["pool"].k, st["pool"].v, st["pool"].ks, st["pool"].vs) if t is not None]
    w0 = st["w"].clone()

    def reset():
        for t, b in zip((st["pool"].k, st["pool"].v, st["pool"].ks, st["pool"].vs), start):
            t.view(torch.uint8).copy_(b)
        st["w"].copy_(w0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(st)
    for lens, seed in (([200 + n, 237 + n, 274 + n], 1), ([n, 90, 101 + n], 2), ([n + 3, n, 250], 3)):
        st["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        st["off"].copy_(torch.tensor([seed, 0, 5], dtype=torch.int32))
        st["x"].copy_(_rand(st["x"].shape, torch.bfloat16, 300 + seed))
        reset()
        graph.replay()
        got = [t.clone() for t in captured]
        reset()
        want = _step(st)
        assert _same(got, want), lens
    vdx.sync_check()


@pytest.mark.parametrize("bits", [16, 8])
def test_two_streams_at_once_keep_apart(bits):
    states = [_state(bits, 20 + i, n) for i, n in enumerate((1, 60))]
    alone = [_step(_state(bits, 20 + i, n), sync=True) for i, n in enumerate((1, 60))]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = []
    for st, stream in zip(states, streams):
        with torch.cuda.stream(stream):
            got.append(_step(st))
    torch.cuda.synchronize()
    vdx.sync_check()
    for a, b in zip(got, alone):
        assert _same(a, b)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [1, 140])
def test_offsets_past_32_bits(bits, n):
    # pages so far apart that byte and element offsets pass 2^31; eviction from the first pages to the last ones
    dt, H, d, page, far = torch.bfloat16, 2, 128, 128, 1 << 31
    pages = 4
    flat = [torch.zeros(3 * far + 2 * page * H * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    if bits == 8:
        k, v = (f.as_strided((pages, page, H, d), (far, H * d, d, 1)).view(CODE) for f in flat)
        ks, vs = (torch.zeros(pages, 8, H, dtype=torch.uint8, device="cuda").view(SCALE) for _ in range(2))
    else:
        k, v = (f.view(dt).as_strided((pages, page, H, d), (far // 2, H * d, d, 1)) for f in flat)
        ks = vs = None
    table = torch.tensor([[3, 0], [2, 1]], dtype=torch.int32, device="cuda")
    lens = [150, 200]
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = _rand((350, 2, H, d), dt, 3)
    cache = vdx.PagedKV(k, v, table, ks, vs)
    vdx.rope3d_append(None, first[:, 0], first[:, 1], cache, cu_of(lens), kv_len, (999, 1, 1))
    x = _rand((2 * n, 3 * H, d), dt, 4)
    q = vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], cache, cu_of([n, n]), kv_len, (999, 1, 1))
    out, lse = vdx.paged_attn(q, cache, cu_of([n, n]), kv_len, max_q=n, causal_block=1)
    w = torch.zeros(2, H, 256, device="cuda")
    vdx.paged_attn_weights(q, cache, cu_of([n, n]), kv_len, lse, w, max_q=n, causal_block=1)
    vdx.sync_check()
    pool = Pool.__new__(Pool)
    pool.bits, pool.page, pool.k, pool.v, pool.ks, pool.vs = bits, page, k, v, ks, vs
    for s, L in enumerate(lens):
        rows = slice(s * n, (s + 1) * n)
        kk, vv = pool.values(table, s, L, "k"), pool.values(table, s, L, "v")
        (check_attention if bits == 16 else check_attention8)(out[rows], lse[:, rows], attend(q[rows], kk, vv, limits(n, L, 1)), dt)
        add, b = weigh(q[rows], kk, limits(n, L, 1), lse[:, rows])
        old = max(0, L - n)
        assert bool(((w[s, :, :L].double() - add).abs() <= b + 2.0 ** -22 * add).all()) and old >= 0
    # sequence 1's pages hold what stays of sequence 0: page 1 is free for it once sequence 1 is gone
    one = vdx.PagedKV(k, v, table[:1], ks, vs)
    into = vdx.PagedKV(k, v, torch.tensor([[1]], dtype=torch.int32, device="cuda"), ks, vs)
    full = [pool.values(table, 0, 150, a) for a in "kv"]
    left = vdx.paged_evict(one, w[:1], kv_len[:1].clone(), 100, into, recent=10)
    vdx.sync_check()
    idx, heads = left.index[0].long().T, torch.arange(H, device="cuda")[None]
    for a, x in zip("kv", full):
        got, want = pool.values(into.page_table, 0, 100, a), x[idx, heads]
        assert bool(((got - want).abs() <= (0 if bits == 16 else 2.0 ** -10) * powers(least_exponent(want.abs().amax((0, 2))))[None, :, None]).all())


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("g,d", [(128, 64), (100, 128), (7, 64), (64, 128)])
def test_groups_of_many_heads(bits, g, d):
    dt, page, lens, news = torch.bfloat16, 64, [150, 77], [3, 2]
    if bits == 8:
        c = Paged8(d, 1, page, lens, 5)
        cache, values = c.cache(vdx), lambda s: (c.get(c.k, c.k_scale, s), c.get(c.v, c.v_scale, s))
    else:
        from streaming_ref import Paged
        c = Paged(dt, d, 1, page, lens, 5)
        cache, values = vdx.PagedKV(c.k, c.v, c.table), lambda s: tuple(x.double() for x in c.get(s))
    q = _rand((5, g, d), dt, 6, 0.7)
    w = torch.zeros(2, 1, 150, device="cuda")
    out, lse = vdx.paged_attn(q, cache, cu_of(news), c.kv_len, max_q=3, causal_block=1)
    vdx.paged_attn_weights(q, cache, cu_of(news), c.kv_len, lse, w, max_q=3, causal_block=1)
    vdx.sync_check()
    at = 0
    for s, n in enumerate(news):
        k, v = values(s)
        lim = limits(n, lens[s], 1)
        (check_attention if bits == 16 else check_attention8)(out[at:at + n], lse[:, at:at + n], attend(q[at:at + n], k, v, lim), dt)
        add, b = weigh(q[at:at + n], k, lim, lse[:, at:at + n])
        assert bool(((w[s, :, :lens[s]].double() - add).abs() <= b + 2.0 ** -22 * add).all())
        at += n


def test_nan_rows_and_stale_slots_stay_where_they_are():
    # a row of NaN queries among others, in each kernel; slots past a length hold NaN codes and scales (Paged8)
    d, H, dt = 128, 2, torch.bfloat16
    c = Paged8(d, H, 16, [100, 333], seed=5)
    for n in (2, 60):
        q = _rand((2 * n, H, d), dt, 6)
        q[1, 0] = math.nan
        out, lse = vdx.paged_attn(q, c.cache(vdx), cu_of([n, n]), c.kv_len, max_q=n)
        w = torch.zeros(2, H, 400, device="cuda")
        vdx.paged_attn_weights(q, c.cache(vdx), cu_of([n, n]), c.kv_len, lse, w, max_q=n)
        vdx.sync_check()
        assert bool(out[1, 0].isnan().all()) and bool(lse[0, 1].isnan()) and int(out.isnan().sum()) == d and int(lse.isnan().sum()) == 1
        assert bool(w[0, 0, :100].isnan().all()) and not bool(w[0, 0, 100:].isnan().any()) and not bool(w[0, 1].isnan().any())
        assert not bool(w[1].isnan().any())


def test_calls_on_8_bits_keep_no_memory():
    st = _state(8, 30, 1)
    _step(st)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(20):
        _step(st)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
