"""Eviction from sequences whose weights take a block of the selection more than one step of its ordered walk (4096 weights
a step, eight blocks a head), up to the longest that is taken."""
import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from kv8_ref import Paged8, stay
from streaming_ref import Paged

pytestmark = pytest.mark.gpu

D, PAGE, PAGE_TO = 64, 4096, 256
KMAX = 393216


def _into(H, keep, bits):
    pages = -(-keep // PAGE_TO)
    table = torch.randperm(pages + 2, device="cuda")[:pages].int()[None].contiguous()
    shape = (pages + 2, PAGE_TO, H, D)
    if bits == 16:
        k, v = (torch.zeros(shape, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        return vdx.PagedKV(k, v, table)
    k, v = (torch.zeros(shape, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros((pages + 2, PAGE_TO // 16, H), device="cuda", dtype=torch.uint8).view(torch.float8_e8m0fnu) for _ in range(2))
    return vdx.PagedKV(k, v, table, ks, vs)


def _check(c, into, w, first, got, L, keep, recent, bits):
    H = c.Hkv
    left = min(L, keep)
    assert got.kv_len.tolist() == [left] and got.pos_offset.tolist() == [L - left]
    slot = torch.arange(left, device="cuda")
    page = into.page_table[0].long()[slot // PAGE_TO]
    for h in range(H):
        kept = torch.tensor(stay(first[0, h], L, keep, recent), device="cuda")
        assert torch.equal(got.index[0, h, :left].long(), kept) and bool((got.index[0, h, left:] == -1).all()), h
        assert torch.equal(got.weights[0, h, :left], first[0, h][kept])
        if bits == 16:
            k, v = c.get(0, L)
            assert torch.equal(into.k[page, slot % PAGE_TO, h], k[kept, h]) and torch.equal(into.v[page, slot % PAGE_TO, h], v[kept, h])
    if bits == 8:
        kept = torch.stack([torch.tensor(stay(first[0, h], L, keep, recent), device="cuda") for h in range(H)], 1)
        heads = torch.arange(H, device="cuda")[None]
        want = Paged8(D, H, PAGE_TO, [0], 0, width=into.page_table.shape[1], spare=into.page_table.shape[1])
        want.table = into.page_table
        for codes, scales, to, to_scale in ((c.k, c.k_scale, into.k, into.k_scale), (c.v, c.v_scale, into.v, into.v_scale)):
            bits_, sc = torch.zeros_like(to.view(torch.uint8)), torch.zeros_like(to_scale.view(torch.uint8))
            want.put(bits_, sc, 0, 0, c.get(codes, scales, 0, L)[kept, heads])
            assert torch.equal(to.view(torch.uint8), bits_) and torch.equal(to_scale.view(torch.uint8), sc)


def _run(L, H, keep, recent, w, bits=16, in_place=False):
    c = (Paged(torch.bfloat16, D, H, PAGE, [L], 501) if bits == 16 else Paged8(D, H, PAGE, [L], 501))
    cache = vdx.PagedKV(c.k, c.v, c.table) if bits == 16 else c.cache(vdx)
    into, first = _into(H, keep, bits), w.clone()
    got = vdx.paged_evict(cache, w, c.kv_len, keep, into, recent=recent, max_kv=L, weights_out=w if in_place else None)
    vdx.sync_check()
    assert torch.equal(w[:, :, keep:], first[:, :, keep:]) and (in_place or torch.equal(w, first))
    _check(c, into, w, first, got, L, keep, recent, bits)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("in_place", [False, True])
def test_runs_of_two_steps(bits, in_place):
    g = torch.Generator(device="cuda").manual_seed(502)
    _run(40003, 2, 20011, 777, torch.rand(1, 2, 40003, generator=g, device="cuda"), bits, in_place)


# 33000 keys are runs of 4128: ties around the 4096th weight of the first run, of the sixth, and over the end of the second
@pytest.mark.parametrize("more", [0, 1, 7, 8, 9, 20, 40, 47, 60, 75, 80])
def test_ties_on_both_sides_of_a_step(more):
    L, run, heavy, recent = 33000, 4128, 500, 50
    ties = [i for at in (4096, 2 * run, 5 * run + 4096) for i in range(at - 8, at + 20)]
    g = torch.Generator(device="cuda").manual_seed(503)
    w = torch.rand(1, 3, L, generator=g, device="cuda")
    for h in range(3):
        spots = [i for i in torch.randperm(L - recent, generator=torch.Generator().manual_seed(504 + h)).tolist() if i not in set(ties)]
        w[0, h, spots[:heavy]] = 10 + torch.rand(heavy, generator=g, device="cuda")
    w[:, :, ties] = 5.0
    _run(L, 3, heavy + more + recent, recent, w)


@pytest.mark.parametrize("kind", ["spread", "alike"])
def test_the_longest_sequence(kind):
    g = torch.Generator(device="cuda").manual_seed(505)
    w = torch.randn(1, 1, KMAX, generator=g, device="cuda").exp() if kind == "spread" else torch.ones(1, 1, KMAX, device="cuda")
    if kind == "alike":
        w[0, 0, 1000::977] = 2.0
    _run(KMAX, 1, 1500, 11, w)


def test_longer_ones_are_refused():
    c = Paged(torch.bfloat16, D, 1, PAGE, [KMAX + 1], 506)
    cache, w = vdx.PagedKV(c.k, c.v, c.table), torch.zeros(1, 1, KMAX + 1, device="cuda")
    into = _into(1, 100, 16)
    for kw in (dict(), dict(max_kv=KMAX + 1)):
        with pytest.raises(vdx.VdxError, match="393216"):
            vdx.paged_evict(cache, w, c.kv_len, 100, into, **kw)
    vdx.paged_evict(cache, w, c.kv_len, 100, into, max_kv=KMAX)            # taken, and the length clamped
    with pytest.raises(vdx.VdxError, match="kv_len"):
        vdx.sync_check()
