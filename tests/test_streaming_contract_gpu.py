"""Promises of the paged-cache and cross-attention calls, on the GPU, beside the formulas that
test_streaming_gpu.py checks: order in a stream, what is reported, and what is left alone."""
import math

import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from streaming_ref import (SECTIONS, Paged, attend, check_attention, cu_of, limits, rotate, rotate_bound)  # noqa: F401
from test_streaming_gpu import _built, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ order in a stream
@pytest.mark.parametrize("n", [1, 40])
def test_a_bare_chain_of_calls_reads_what_the_call_before_wrote(n):
    # append and attention alternate over the same q, cache and scratch with nothing between them and no
    # synchronisation; the same steps one at a time are the reference
    dt, H, d, page, S, steps = torch.bfloat16, 4, 128, 16, 3, 150
    first = 64 if n == 1 else 0
    width = -(-(first + n * steps) // page)
    xs = _rand((steps, S * n, 3 * H, d), dt, 100)
    lens = (first + n * torch.arange(1, steps + 1, device="cuda", dtype=torch.int32))[:, None].expand(-1, S).contiguous()
    cu, grid = cu_of([n] * S), (first + n * steps, 1, 1)
    results = []
    for alone in (True, False):
        k, v = (torch.zeros(S * width, page, H, d, dtype=dt, device="cuda") for _ in range(2))
        cache = vdx.PagedKV(k, v, torch.arange(S * width, dtype=torch.int32, device="cuda").view(S, width))
        q = torch.zeros(S * n, H, d, dtype=dt, device="cuda")
        outs = torch.zeros(steps, S * n, H, d, dtype=dt, device="cuda")
        lse = torch.zeros(steps, H, S * n, device="cuda")
        top = first + n * steps
        ws = torch.empty(vdx.paged_attn_workspace_bytes(q, cache, cu, lens[0], n, top) + 16, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            x = xs[i]
            vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], cache, cu, lens[i], grid, q_out=q)
            if alone:
                torch.cuda.synchronize()
            vdx.paged_attn(q, cache, cu, lens[i], max_q=n, max_kv=top, causal_block=1, out=outs[i], lse=lse[i], workspace=ws)
            if alone:
                torch.cuda.synchronize()
        vdx.sync_check()
        results.append((outs, lse, k, v))
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 40])
def test_calls_right_behind_kernels_that_rewrite_their_inputs(n):
    # lengths, page table, rows, norm weights and queries are overwritten by kernels queued just ahead of each call
    dt, H, d, page, S, steps = torch.bfloat16, 4, 128, 16, 4, 100
    width = 24
    g = torch.Generator(device="cuda").manual_seed(101)
    xs = _rand((2, S * n, 3 * H, d), dt, 102)
    weights = _rand((2, d), dt, 103)
    lens = torch.tensor([[60, 300, 41, 384], [384, 40, 200, 77]], dtype=torch.int32, device="cuda")
    cus = torch.stack([cu_of([n] * S), cu_of([n - 1, n, n, n])])
    tables = torch.stack([torch.randperm(S * width, generator=g, device="cuda").int().view(S, width) for _ in range(2)])
    k0, v0 = _rand((S * width, page, H, d), dt, 104), _rand((S * width, page, H, d), dt, 105)
    grid = (400, 1, 1)
    results = []
    for alone in (True, False):
        x, w, kv_len, cu, table = (torch.empty_like(t[0]) for t in (xs, weights, lens, cus, tables))
        k, v = k0.clone(), v0.clone()
        cache = vdx.PagedKV(k, v, table)
        outs = torch.zeros(steps, S * n, H, d, dtype=dt, device="cuda")
        rot = torch.zeros(steps, S * n, H, d, dtype=dt, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            for t, src in ((x, xs), (w, weights), (kv_len, lens), (cu, cus), (table, tables)):
                torch.add(src[i & 1], 0, out=t)
            if alone:
                torch.cuda.synchronize()
            vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], cache, cu, kv_len, grid, q_norm=w, k_norm=w, q_out=rot[i])
            torch.add(lens[(i + 1) & 1], 0, out=kv_len)             # attention over other lengths than were appended to
            if alone:
                torch.cuda.synchronize()
            vdx.paged_attn(rot[i], cache, cu, kv_len, max_q=n, max_kv=384, out=outs[i])
            if alone:
                torch.cuda.synchronize()
        vdx.sync_check()
        results.append((rot, outs, k, v))
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------ append: what is reported
@pytest.mark.parametrize("rows", [8, 600])
@pytest.mark.parametrize("bad", ["past the rows", "negative", "decreasing", "decreasing behind the rows"])
def test_append_reports_ranges_that_are_none(rows, bad):
    dt, H, d = torch.bfloat16, 2, 64
    lens = [rows + 20, rows + 20]
    cu = {"past the rows": [0, rows + 2, rows + 2], "negative": [-2, rows // 2, rows // 2],
          "decreasing": [0, rows, rows // 2], "decreasing behind the rows": [0, 0, -1]}[bad]
    # the first sequence of "decreasing" has a good range: its tokens go where they belong
    good = rows if bad == "decreasing" else 0
    c = Paged(dt, d, H, 16, lens, seed=110)
    k0, v0 = c.k.clone(), c.v.clone()
    q, k, v = (_rand((rows, H, d), dt, 111 + i) for i in range(3))
    out = torch.full_like(q, 5.0)
    cache, grid = vdx.PagedKV(c.k, c.v, c.table), (2000, 1, 1)
    vdx.rope3d_append(q, k, v, cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), c.kv_len, grid, q_out=out)
    with pytest.raises(vdx.VdxError, match="cu or kv_len broke a bound"):
        vdx.sync_check()
    assert bool((out[good:] == 5.0).all())
    written = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    pos = torch.arange(20, 20 + good, device="cuda")
    if good:
        written[c.slots(0, pos)] = True
        assert torch.equal(c.v[c.slots(0, pos)], v)
    for now, was in ((c.k, k0), (c.v, v0)):
        assert torch.equal(now[~written].view(torch.int16), was[~written].view(torch.int16))
    # rows behind the last sequence are no mistake
    vdx.rope3d_append(q, k, v, cache, cu_of([3, 2]), c.kv_len, grid, q_out=out)
    vdx.sync_check()


@pytest.mark.parametrize("n", [8, 700])
def test_two_rows_for_one_slot_leave_pieces_of_either(n):
    # two sequences over the same pages at the same indices: every 16 bytes are one row's, every other slot is as it was
    dt, H, d = torch.bfloat16, 3, 64
    c = Paged(dt, d, H, 16, [n + 5, n + 5], seed=120)
    c.table[1] = c.table[0]
    before = c.k.clone(), c.v.clone()
    k, v = (_rand((2 * n, H, d), dt, 121 + i) for i in range(2))
    vdx.rope3d_append(None, k, v, vdx.PagedKV(c.k, c.v, c.table), cu_of([n, n]), c.kv_len, (2000, 1, 1), SECTIONS[d])
    vdx.sync_check()
    pos = torch.arange(5, 5 + n, device="cuda")
    slots = c.slots(0, pos)
    got = c.v[slots].view(n, H, d // 8, 8)
    a, b = v[:n].view(n, H, d // 8, 8), v[n:].view(n, H, d // 8, 8)
    assert bool(((got == a).all(-1) | (got == b).all(-1)).all())
    errs = []
    for x in (k[:n], k[n:]):
        ref = rotate(x, pos, (2000, 1, 1), SECTIONS[d], 10000.0)
        errs.append(((c.k[slots].double() - ref).abs() <= rotate_bound(ref, dt)).view(n, H, d // 8, 8).all(-1))
    assert bool((errs[0] | errs[1]).all())
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    touched[slots] = True
    for now, was in zip((c.k, c.v), before):
        assert torch.equal(now[~touched].view(torch.int16), was[~touched].view(torch.int16))


# ------------------------------------------------------------------------- frame-causal masks and dropped pages
def _offset_limits(n, length, block, off):
    p = torch.arange(length - n, length, device="cuda")
    lim = (torch.div(p + off, block, rounding_mode="floor") + 1) * block - off
    return torch.where(p < 0, torch.zeros_like(p), lim.clamp(0, length))


@pytest.mark.parametrize("block", [1, 7, 100, 1560, 2 ** 31 - 1])
@pytest.mark.parametrize("news,lens,offs", [
    ([1, 3, 2], [50, 300, 7], [0, 93, 640]),                       # the few-row kernel
    ([1], [20000], [1111]),                                        # its splits, joined through scratch
    ([40, 300, 0, 129], [90, 700, 5, 129], [256, 99, 13, 5]),      # tiles
    ([200, 1], [3000, 2000], [1559, 2 ** 31 - 1]),                 # split tiles; the largest offset
    ([5, 60], [3, 50], [3, 1600]),                                 # more rows than keys: negative indices see nothing
])
def test_blocks_are_counted_from_grid_token_zero(news, lens, offs, block):
    dt, H, d, page = torch.bfloat16, 2, 64, 32
    c = Paged(dt, d, H, page, lens, seed=130)
    q = _rand((sum(news), H, d), dt, 131, 1.5)
    out, lse = vdx.paged_attn(q, vdx.PagedKV(c.k, c.v, c.table), cu_of(news), c.kv_len, max_q=max(news), max_kv=max(lens),
                              causal_block=block, pos_offset=torch.tensor(offs, dtype=torch.int32, device="cuda"))
    vdx.sync_check()
    at = 0
    for s, (n, length, off) in enumerate(zip(news, lens, offs)):
        k, v = c.get(s)
        check_attention(out[at:at + n], lse[:, at:at + n], attend(q[at:at + n], k, v, _offset_limits(n, length, block, off)), dt,
                        f"sequence {s}: {n} of {length}, offset {off}")
        at += n


def test_negative_offsets_and_no_mask():
    # an offset below 0 (tokens that the cache keeps before the grid's first): blocks are counted downwards too
    dt, H, d = torch.float16, 2, 64
    c = Paged(dt, d, H, 16, [90, 200], seed=132)
    q = _rand((42, H, d), dt, 133, 1.5)
    cache, off = vdx.PagedKV(c.k, c.v, c.table), torch.tensor([-30, -101], dtype=torch.int32, device="cuda")
    for block in (1, 24):
        out, lse = vdx.paged_attn(q, cache, cu_of([2, 40]), c.kv_len, max_q=40, max_kv=200, causal_block=block, pos_offset=off)
        for s, rows, length in ((0, slice(0, 2), 90), (1, slice(2, 42), 200)):
            k, v = c.get(s)
            ref = attend(q[rows], k, v, _offset_limits(rows.stop - rows.start, length, block, int(off[s])))
            check_attention(out[rows], lse[:, rows], ref, dt)
    a = vdx.paged_attn(q, cache, cu_of([2, 40]), c.kv_len, max_q=40, max_kv=200, pos_offset=off)
    b = vdx.paged_attn(q, cache, cu_of([2, 40]), c.kv_len, max_q=40, max_kv=200)
    vdx.sync_check()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_dropping_pages_inside_a_frame_changes_only_what_is_gone():
    # pages of 16 tokens, frames of 54: the first pages leave the table, the new frame still sees whole frames
    dt, H, d, page, frame, frames = torch.bfloat16, 2, 128, 16, 54, 4
    grid = (frames + 1, 6, 9)
    n, total = frame + 20, frame * frames + 20                    # the chunk: the last frame and part of the next
    width = -(-total // page)
    k, v = (torch.full((width, page, H, d), math.nan, dtype=dt, device="cuda") for _ in range(2))
    x = _rand((total, 3 * H, d), dt, 134)
    table = torch.arange(width, dtype=torch.int32, device="cuda").view(1, -1)
    rot = vdx.rope3d_append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], vdx.PagedKV(k, v, table), cu_of([total]),
                            torch.tensor([total], dtype=torch.int32, device="cuda"), grid, SECTIONS[d])
    kk, vv = k.view(-1, H, d)[:total], v.view(-1, H, d)[:total]
    for gone in (1, 5):
        drop = gone * page
        cache = vdx.PagedKV(k, v, table[:, gone:].contiguous())
        lens, off = (torch.tensor([t], dtype=torch.int32, device="cuda") for t in (total - drop, drop))
        again = vdx.rope3d_append(x[-n:, :H], x[-n:, H:2 * H], x[-n:, 2 * H:], cache, cu_of([n]), lens, grid, SECTIONS[d],
                                  pos_offset=off)
        assert torch.equal(again, rot[-n:])
        out, lse = vdx.paged_attn(again, cache, cu_of([n]), lens, max_q=n, causal_block=frame, pos_offset=off)
        vdx.sync_check()
        p = torch.arange(total - n, total, device="cuda")
        lim = ((torch.div(p, frame, rounding_mode="floor") + 1) * frame).clamp(max=total) - drop
        check_attention(out, lse, attend(rot[-n:], kk[drop:], vv[drop:], lim), dt, f"{gone} pages gone")


# ------------------------------------------------------------------------------------ autograd
def _small(seed=140):
    dt = torch.bfloat16
    c = Paged(dt, 64, 2, 16, [40, 9], seed=seed)
    x, text = _rand((2, 2, 64), dt, seed + 1), _rand((1, 50, 2, 64), dt, seed + 2)
    return c, vdx.PagedKV(c.k, c.v, c.table), x, cu_of([1, 1]), text


def test_tangents_and_transforms_are_refused():
    import torch.autograd.forward_ad as fw
    c, cache, x, cu, text = _small()
    calls = [lambda t: vdx.rope3d_append(t, x, x, cache, cu, c.kv_len, (50, 1, 1)),
             lambda t: vdx.rope3d_append(x, t, x, cache, cu, c.kv_len, (50, 1, 1)),
             lambda t: vdx.rope3d_append(x, x, t, cache, cu, c.kv_len, (50, 1, 1)),
             lambda t: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, 1, 1), k_norm=t[0, 0]),
             lambda t: vdx.paged_attn(t, cache, cu, c.kv_len),
             lambda t: vdx.cross_attn(t[None], text, text)[0][0],
             lambda t: vdx.cross_attn(text, t[None], t[None])[0]]
    for i, f in enumerate(calls):
        with fw.dual_level():
            with pytest.raises(vdx.VdxError, match="forward"):
                f(fw.make_dual(x, torch.ones_like(x)))
                pytest.fail(f"call {i} took a tangent")
        with pytest.raises(vdx.VdxError, match="forward"):
            torch.func.jvp(lambda t: f(t), (x,), (torch.ones_like(x),))
        with pytest.raises(vdx.VdxError, match="transform"):
            torch.func.vmap(f)(x[None])
        f(x)
    with pytest.raises(vdx.VdxError, match="gradient"):
        vdx.paged_attn(x, cache, cu, c.kv_len, lse=torch.zeros(2, 2, device="cuda", requires_grad=True))
    vdx.sync_check()


def test_autograd_sees_what_the_calls_write():
    # a tensor that autograd saved and a call then overwrote must not be used for a gradient
    c, cache, x, cu, text = _small(150)
    w = torch.ones((), device="cuda", requires_grad=True)
    q_out, out, lse = torch.empty_like(x), torch.empty_like(x), torch.empty(2, 2, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    text_out = torch.empty_like(text)
    with torch.no_grad():
        for t in (q_out, out, lse, text_out):
            t.zero_()
    calls = [(lambda: vdx.rope3d_append(x, x, x, cache, cu, c.kv_len, (50, 1, 1), q_out=q_out), [c.k, c.v, q_out], [x, c.table, cu]),
             (lambda: vdx.rope3d_append(None, x, x, cache, cu, c.kv_len, (50, 1, 1)), [c.k, c.v], [x]),
             (lambda: vdx.paged_attn(x, cache, cu, c.kv_len, out=out, lse=lse, workspace=ws), [out, lse, ws], [x, c.k, c.v]),
             (lambda: vdx.cross_attn(text, text, text, out=text_out), [text_out], [text])]
    for call, writes, reads in calls:
        saved = [(t, (w * t.detach()).sum()) for t in writes + reads if t.dtype.is_floating_point]   # saves t for w's gradient
        before = [t._version for t in writes + reads]
        call()
        now = [t._version for t in writes + reads]
        assert all(b > a for a, b in zip(before[:len(writes)], now)) and now[len(writes):] == before[len(writes):]
        for t, y in saved:
            if any(t is o for o in writes):
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    y.backward()
            else:
                y.backward()
    with torch.inference_mode():                                   # tensors without a version
        a, b = torch.zeros_like(c.k), torch.zeros_like(c.v)
        o = torch.empty_like(x)
    vdx.rope3d_append(x, x, x, vdx.PagedKV(a, b, c.table), cu, c.kv_len, (50, 1, 1), q_out=o)
    vdx.sync_check()
    assert bool((b != 0).any())


# ------------------------------------------------------------------------------------ what is refused
def test_workspace_sizes_of_calls_that_are_refused():
    dt = torch.bfloat16
    c, cache, x, cu, text = _small(160)
    wide = torch.zeros(2, 258, 64, dtype=dt, device="cuda")       # 129 query heads to a head of the cache
    odd = torch.zeros(2, 3, 64, dtype=dt, device="cuda")
    for f in (lambda: vdx.paged_attn_workspace_bytes(wide, cache, cu, c.kv_len), lambda: vdx.paged_attn_workspace_bytes(odd, cache, cu, c.kv_len),
              lambda: vdx.paged_attn_workspace_bytes(x, cache, None, c.kv_len),
              lambda: vdx.cross_attn_workspace_bytes(text[..., :32], text[..., :32], text[..., :32]),
              lambda: vdx.cross_attn_workspace_bytes(text, text[:, :, :1].expand(-1, -1, 3, -1), text[:, :, :1].expand(-1, -1, 3, -1))):
        with pytest.raises(vdx.VdxError):
            f()
    assert vdx.paged_attn_workspace_bytes(x, cache, cu, c.kv_len, 1, 40) == 0
    assert vdx.cross_attn_workspace_bytes(text[:, :0], text, text) == 0
    long = torch.zeros(1, 30000, 2, 64, dtype=dt, device="cuda")
    assert vdx.cross_attn_workspace_bytes(text[:, :1], long, long) > 0


# ------------------------------------------------------------------------------------ the check of what was reported
def test_a_check_costs_one_read_until_the_streaming_calls_are_used():
    # in a process of its own: before any of these calls, vdx_sync_check reads the self-attention's word alone
    # (one synchronous copy of 4 bytes, as .item() makes one; it takes 1.0 to 1.5 of that, four copies 4)
    import os
    import subprocess
    import sys
    code = """
import sys, time, torch
import video_diffusion_transformer_rope_gb300 as vdx
x = torch.zeros(1, device="cuda")
def best(f):
    for _ in range(20):
        f()
    t = []
    for _ in range(9):
        a = time.perf_counter()
        for _ in range(50):
            f()
        t.append(time.perf_counter() - a)
    return min(t)
print(best(vdx.sync_check) / best(lambda: (torch.cuda.current_stream().synchronize(), x.item())))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert float(r.stdout) < 2.5, r.stdout


@pytest.mark.parametrize("at", [151, 250, 299])
def test_append_looks_at_the_range_of_every_sequence(at):
    # 300 sequences of which one has rows; a later range runs backwards, where no row of the call looks
    S, H, d = 300, 1, 64
    dt = torch.bfloat16
    k = torch.zeros(S, 16, H, d, dtype=dt, device="cuda")
    cache = vdx.PagedKV(k, k.clone(), torch.arange(S, dtype=torch.int32, device="cuda").view(S, 1))
    x = _rand((4, H, d), dt, 170)
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    cu[150:] = 4
    kv_len = torch.full((S,), 4, dtype=torch.int32, device="cuda")
    vdx.rope3d_append(None, x, x, cache, cu, kv_len, (16, 1, 1))
    vdx.sync_check()
    assert torch.equal(cache.v[149, :4], x)
    cu[at + 1:] = 3
    vdx.rope3d_append(None, x, x, cache, cu, kv_len, (16, 1, 1))
    with pytest.raises(vdx.VdxError, match="cu or kv_len broke a bound"):
        vdx.sync_check()
