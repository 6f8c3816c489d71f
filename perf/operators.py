"""Measured cases of the operators that stand beside the 3D-RoPE self-attention: appending a chunk of new tokens
to a paged key/value cache (per-head norms and the rotary positions applied on the way), attention of such a
chunk over the cache, and cross attention to an encoder's states.

Head counts, head dimensions, grids, rotary sections and theta are those of the Wan-shaped workloads in
video_diffusion_transformer_rope_gb300/configs.py (12 and 40 heads of 128, 30x52 and 45x80 latent frames, 21 of
them; the tiny one has 4 heads of 64); 512 is the text length and 257 the image length of such models' encoders.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
SECTIONS = {128: (44, 42, 42), 64: (24, 20, 20)}
THETA = 10000.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases
def _append(name, **kw):
    return dict(dict(name=name, op="append", dtype="bf16", d=128, seqs=1, heads=12, kv_heads=12, new_min=1, new_max=1,
                     ctx_min=0, ctx_max=0, page=128, frames=1024, rows=30, cols=52, norm=True, offset=0, layout=1), **kw)


def _paged(name, **kw):
    return dict(dict(name=name, op="paged", dtype="bf16", d=128, seqs=1, heads=12, kv_heads=12, new_min=1, new_max=1,
                     ctx_min=0, ctx_max=0, page=128, block=0, layout=1), **kw)


def _cross(name, **kw):
    return dict(dict(name=name, op="cross", dtype="bf16", d=128, batch=2, heads=12, kv_heads=12, n=1, m=512,
                     ragged=False, layout=1), **kw)


def listed():
    return [
        # one new token for each of eight sequences: the smallest append, all latency
        _append("append_token", seqs=8, ctx_min=100, ctx_max=2000, page=16, rows=1, cols=1, frames=4096),
        # one 480p latent frame for both halves of a guided pair, a page per frame, positions past the cache's
        # own indices (older frames were dropped)
        _append("append_frame_480p", seqs=2, new_min=1560, new_max=1560, ctx_min=3120, ctx_max=3120, page=1560, offset=46800),
        # three 720p latent frames for a guided pair: the largest append, all bandwidth
        _append("append_chunk_720p", seqs=2, heads=40, kv_heads=40, new_min=10800, new_max=10800, ctx_min=3600, ctx_max=3600,
                page=128, rows=45, cols=80),
        # ragged prompts with grouped heads, half precision, no norm
        _append("append_ragged_fp16", dtype="fp16", d=64, seqs=13, kv_heads=4, new_min=1, new_max=301, ctx_min=0, ctx_max=500,
                page=32, norm=False, rows=1, cols=1, frames=4096),
        # a few sequences at one token each over short caches: latency
        _paged("paged_token_small", seqs=4, ctx_min=64, ctx_max=1000, page=16),
        # many sequences at one token each over long caches with grouped heads: reading the cache
        _paged("paged_token_large", seqs=48, heads=40, kv_heads=8, ctx_min=8000, ctx_max=32759, page=64),
        # a 480p latent frame over 21 frames, both halves of a guided pair, a page per frame
        _paged("paged_frame_480p", seqs=2, new_min=1560, new_max=1560, ctx_min=31200, ctx_max=31200, page=1560, block=1560),
        # a 720p latent frame over 21 frames: the largest chunk
        _paged("paged_frame_720p", heads=40, kv_heads=40, new_min=3600, new_max=3600, ctx_min=72000, ctx_max=72000, page=128,
               block=3600),
        # ragged chunks, every token after the ones before it, grouped heads, half precision
        _paged("paged_ragged_fp16", dtype="fp16", d=64, seqs=9, kv_heads=4, new_min=1, new_max=500, ctx_min=0, ctx_max=3000,
               page=16, block=1),
        # the tiny workload's grid against a short prompt: latency
        _cross("cross_tiny_fp16", dtype="fp16", d=64, batch=1, heads=4, kv_heads=4, n=192, m=77),
        # 480p latents of a guided pair against their two prompts, of different lengths
        _cross("cross_480p", n=32760, ragged=True),
        # 720p latents against full-length text: the largest
        _cross("cross_720p", heads=40, kv_heads=40, n=75600),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_once(rng):
    heads, kv = rng.choice([(12, 12), (40, 40), (12, 4), (40, 8), (4, 4), (40, 40), (12, 12), (12, 1)])
    common = dict(dtype=rng.choice(["bf16", "bf16", "fp16"]), d=rng.choice([128, 128, 64]), heads=heads, kv_heads=kv,
                  layout=rng.randrange(1 << 30))
    op = rng.choice(["append", "paged", "paged", "cross", "cross"])
    if op == "cross":
        return _cross("", batch=rng.randint(1, 4), n=_log(rng, 1, 75600), m=_log(rng, 1, 1024), ragged=rng.random() < 0.5, **common)
    page = rng.choice([16, 32, 64, 128, 200, 1560, 3600])
    new = _log(rng, 1, 10800 if op == "append" else 3600)
    new_min = rng.choice([1, max(1, new // 2), new])
    ctx = _log(rng, 1, 4000 if op == "append" else 72000)
    ctx_min = rng.choice([0, ctx // 2, ctx])
    seqs = _log(rng, 1, 64)
    ranges = dict(seqs=seqs, new_min=new_min, new_max=new, ctx_min=ctx_min, ctx_max=ctx, page=page)
    if op == "append":
        rows, cols, frames = rng.choice([(30, 52, 1024), (45, 80, 1024), (1, 1, 32768)])
        return _append("", rows=rows, cols=cols, frames=frames, norm=rng.random() < 0.5, offset=rng.choice([0, 0, 1560, 14400]),
                       **ranges, **common)
    return _paged("", block=rng.choice([0, 1, 1560, 3600]), **ranges, **common)


_CAP = {}


def draw(rng):
    if not _CAP:
        for c in listed():
            w, cap = work(c), _CAP.setdefault(c["op"], {"bytes": 0, "flops": 0, "held": 0})
            cap["bytes"], cap["flops"] = max(cap["bytes"], w["bytes"]), max(cap["flops"], w["flops"])
            cap["held"] = max(cap["held"], _held(c))
    while True:
        c = _draw_once(rng)
        w, cap = work(c), _CAP[c["op"]]
        if w["bytes"] <= cap["bytes"] and w["flops"] <= cap["flops"] and _held(c) <= cap["held"]:
            del c["name"]
            return c


# ------------------------------------------------------------------------------------------------ shapes
def _lengths(case):
    """New tokens and cached tokens before them, for each sequence: part of the case, not of the seed."""
    r = random.Random(case["layout"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["seqs"])]
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    return new, ctx


def _key_lengths(case):
    r = random.Random(case["layout"])
    return [r.randint(max(1, case["m"] // 4), case["m"]) if case["ragged"] else case["m"] for _ in range(case["batch"])]


def _pages(case):
    new, ctx = _lengths(case)
    return [-(-(a + b) // case["page"]) for a, b in zip(new, ctx)]


def _held(case):
    """Bytes of the cache that a case keeps (nothing for cross attention)."""
    if case["op"] == "cross":
        return 0
    return 4 * sum(_pages(case)) * case["page"] * case["kv_heads"] * case["d"]


def _visible(n, length, block):
    """Visible (row, key) pairs of a chunk of the last n of `length` tokens."""
    if block == 0:
        return n * length
    total, i = 0, length - n
    while i < length:                                    # rows of one block see the same keys
        last = min(length, (i // block + 1) * block)
        total += (last - i) * last
        i = last
    return total


def work(case):
    hq, hk, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "append":
        n = sum(_lengths(case)[0])
        return {"bytes": 2 * 2 * n * (hq + 2 * hk) * d, "flops": (10 if case["norm"] else 6) * n * (hq + hk) * d}
    if case["op"] == "paged":
        new, ctx = _lengths(case)
        pairs = sum(_visible(n, n + c, case["block"]) for n, c in zip(new, ctx))
        keys = sum(n + c for n, c in zip(new, ctx))
        return {"bytes": 2 * 2 * sum(new) * hq * d + 4 * sum(new) * hq + 2 * 2 * keys * hk * d, "flops": 4 * d * hq * pairs}
    keys = sum(_key_lengths(case))
    rows = case["batch"] * case["n"] * hq
    return {"bytes": 2 * 2 * rows * d + 4 * rows + 2 * 2 * keys * hk * d, "flops": 4 * d * hq * case["n"] * keys}


# ------------------------------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    """Tensors of a case, from the seed alone: activations of about unit variance with a few strong channels (as
    projections give them), normalised queries with a gain that makes attention moderately peaked."""
    dev, dt = torch.device("cuda"), DT[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    hq, hk, d = case["heads"], case["kv_heads"], case["d"]

    def draw_tensor(*shape, gain=1.0, chunk=1 << 28):
        out = torch.empty(shape, dtype=dt, device=dev)
        flat = out.view(-1)
        for i in range(0, flat.numel(), chunk):
            part = flat[i:i + chunk]
            part.copy_(torch.randn(part.shape, generator=g, device=dev, dtype=torch.float32).mul_(gain))
        return out

    if case["op"] == "cross":
        b, n, m = case["batch"], case["n"], case["m"]
        t = {"q": draw_tensor(b, n, hq, d, gain=1.5), "k": draw_tensor(b, m, hk, d), "v": draw_tensor(b, m, hk, d)}
        t["kv_len"] = torch.tensor(_key_lengths(case), dtype=torch.int32, device=dev) if case["ragged"] else None
        return t
    new, ctx = _lengths(case)
    pages = _pages(case)
    total, width, P = sum(pages), max(pages), case["page"]
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((case["seqs"], width), dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(pages):
        table[s, :k] = order[at:at + k]
        at += k
    t = {"k_cache": draw_tensor(total, P, hk, d), "v_cache": draw_tensor(total, P, hk, d), "table": table}
    t["cu"] = torch.tensor([0] + [sum(new[:s + 1]) for s in range(len(new))], dtype=torch.int32, device=dev)
    t["kv_len"] = torch.tensor([a + b for a, b in zip(new, ctx)], dtype=torch.int32, device=dev)
    n = sum(new)
    if case["op"] == "append":
        # one projection's output: q, k and v of a token side by side
        qkv = draw_tensor(n, hq + 2 * hk, d)
        qkv[:, :, d // 3] *= 4
        t["q"], t["k"], t["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        t["offset"] = torch.full((case["seqs"],), case["offset"], dtype=torch.int32, device=dev) if case["offset"] else None
        t["q_norm"] = t["k_norm"] = None
        if case["norm"]:
            t["q_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
            t["k_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
    else:
        t["q"] = draw_tensor(n, hq, d, gain=1.5)
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    st = {"case": case, "t": t}
    if case["op"] != "cross":
        new, ctx = _lengths(case)
        st["new"], st["len"] = new, [a + b for a, b in zip(new, ctx)]
    if own:
        import video_diffusion_transformer_rope_gb300 as vdx
        st["vdx"] = vdx
        if case["op"] != "cross":
            st["cache"] = vdx.PagedKV(t["k_cache"], t["v_cache"], t["table"])
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "paged": _own_paged, "cross": _own_cross}[op](state)
    return {"append": _plain_append, "paged": _plain_paged, "cross": _plain_cross}[op](state)


def _own_append(st):
    c, t = st["case"], st["t"]
    q = st["vdx"].rope3d_append(t["q"], t["k"], t["v"], st["cache"], t["cu"], t["kv_len"], (c["frames"], c["rows"], c["cols"]),
                                sections=SECTIONS[c["d"]], theta=THETA, pos_offset=t["offset"], q_norm=t["q_norm"],
                                k_norm=t["k_norm"], eps=EPS)
    return {"q": q, "k_cache": t["k_cache"], "v_cache": t["v_cache"]}


def _own_paged(st):
    c, t = st["case"], st["t"]
    out, lse = st["vdx"].paged_attn(t["q"], st["cache"], t["cu"], t["kv_len"], max_q=max(st["new"]), max_kv=max(st["len"]),
                                    causal_block=c["block"])
    return {"out": out, "lse": lse}


def _own_cross(st):
    t = st["t"]
    out, lse = st["vdx"].cross_attn(t["q"], t["k"], t["v"], kv_len=t["kv_len"])
    return {"out": out, "lse": lse}


def _plain_append(st):
    c, t = st["case"], st["t"]
    dev, d, n = t["q"].device, c["d"], t["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device=dev), (t["cu"][1:] - t["cu"][:-1]).long(), output_size=n)
    row = torch.arange(n, device=dev) - t["cu"].long()[seq]
    index = t["kv_len"].long()[seq] - (t["cu"][1:] - t["cu"][:-1]).long()[seq] + row
    pos = index + (t["offset"].long()[seq] if t["offset"] is not None else 0)
    area = c["rows"] * c["cols"]
    axes = (pos // area, pos // c["cols"] % c["rows"], pos % c["cols"])
    angle = torch.cat([a.double()[:, None] * THETA ** (-2.0 * torch.arange(s // 2, device=dev, dtype=torch.float64) / s)
                       for a, s in zip(axes, SECTIONS[d])], dim=1)
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()
        even, odd = x[..., 0::2], x[..., 1::2]
        y = torch.empty_like(x)
        y[..., 0::2] = even * cos - odd * sin
        y[..., 1::2] = even * sin + odd * cos
        return y.to(t["q"].dtype)

    page, slot = t["table"].long()[seq, index // c["page"]], index % c["page"]
    t["k_cache"][page, slot] = turn(t["k"], t["k_norm"])
    t["v_cache"][page, slot] = t["v"]
    return {"q": turn(t["q"], t["q_norm"]), "k_cache": t["k_cache"], "v_cache": t["v_cache"]}


def _attend(q, k, v, scale, seen=None, budget=1 << 29):
    """q [n, Hq, d], k and v [L, Hkv, d] -> out [n, Hq, d] and lse [Hq, n], 32 bits; seen [n, L] or None."""
    n, hq, d = q.shape
    length, hk = k.shape[0], k.shape[1]
    g = hq // hk
    out = torch.zeros((hq, n, d), dtype=torch.float32, device=q.device)
    lse = torch.full((hq, n), -math.inf, dtype=torch.float32, device=q.device)
    if length == 0:
        return out.transpose(0, 1), lse
    step = max(1, budget // max(1, g * n * length))
    for a in range(0, hk, step):
        b = min(hk, a + step)
        qh = q[:, a * g:b * g].float().transpose(0, 1).reshape(b - a, g * n, d)
        kh, vh = k[:, a:b].float().transpose(0, 1), v[:, a:b].float().transpose(0, 1)
        s = torch.matmul(qh, kh.transpose(1, 2)) * scale
        if seen is not None:
            s = s.view(b - a, g, n, length).masked_fill_(~seen, -math.inf).view(b - a, g * n, length)
        m = s.amax(dim=-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        total = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p, vh) / torch.where(total == 0, torch.ones_like(total), total)
        out[a * g:b * g] = o.view((b - a) * g, n, d)
        lse[a * g:b * g] = (m + torch.log(total)).view((b - a) * g, n)
    return out.transpose(0, 1), lse


def _seen(n, length, block, dev):
    if block == 0 or n == 0:
        return None
    p = torch.arange(length - n, length, device=dev)
    return torch.arange(length, device=dev)[None, :] < ((p // block + 1) * block)[:, None]


def _plain_paged(st):
    c, t = st["case"], st["t"]
    out = torch.empty_like(t["q"])
    lse = torch.empty((c["heads"], t["q"].shape[0]), dtype=torch.float32, device=out.device)
    at = 0
    for s, (n, length) in enumerate(zip(st["new"], st["len"])):
        pages = t["table"][s, :-(-length // c["page"])].long()
        k = t["k_cache"][pages].reshape(-1, c["kv_heads"], c["d"])[:length]
        v = t["v_cache"][pages].reshape(-1, c["kv_heads"], c["d"])[:length]
        o, l = _attend(t["q"][at:at + n], k, v, c["d"] ** -0.5, _seen(n, length, c["block"], out.device))
        out[at:at + n] = o.to(out.dtype)
        lse[:, at:at + n] = l
        at += n
    return {"out": out, "lse": lse}


def _plain_cross(st):
    c, t = st["case"], st["t"]
    out = torch.empty_like(t["q"])
    lse = torch.empty((c["batch"], c["heads"], c["n"]), dtype=torch.float32, device=out.device)
    for b in range(c["batch"]):
        seen = None
        if t["kv_len"] is not None:
            seen = (torch.arange(c["m"], device=out.device) < t["kv_len"][b])[None, :].expand(c["n"], -1)
        o, l = _attend(t["q"][b], t["k"][b], t["v"][b], c["d"] ** -0.5, seen)
        out[b] = o.to(out.dtype)
        lse[b] = l
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    t = _inputs(case, seed)
    return {"append": _exact_append, "paged": _exact_paged, "cross": _exact_cross}[case["op"]](case, t)


def _exact_append(case, t):
    d, P = case["d"], case["page"]
    new, ctx = _lengths(case)
    dev = t["q"].device
    q_out = torch.empty(t["q"].shape, dtype=torch.float64, device=dev)
    k_cache, v_cache = t["k_cache"].double(), t["v_cache"].double()
    st, sh, sw = SECTIONS[d]
    turns = [THETA ** (-2.0 * j / s) for s in (st, sh, sw) for j in range(s // 2)]
    turns = torch.tensor(turns, dtype=torch.float64, device=dev)

    def rotated(x, weight, positions):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + EPS) * weight.double()
        frame, rest = positions // (case["rows"] * case["cols"]), positions % (case["rows"] * case["cols"])
        coord = torch.cat([frame[:, None].expand(-1, st // 2), (rest // case["cols"])[:, None].expand(-1, sh // 2),
                           (rest % case["cols"])[:, None].expand(-1, sw // 2)], dim=1).double()
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous())
        z = z * torch.polar(torch.ones_like(coord), coord * turns)[:, None, :]
        return torch.view_as_real(z).reshape(x.shape)

    at = 0
    for s, (n, before) in enumerate(zip(new, ctx)):
        index = torch.arange(before, before + n, device=dev)
        where = t["table"][s].long()[index // P] * P + index % P
        positions = index + case["offset"]
        q_out[at:at + n] = rotated(t["q"][at:at + n], t["q_norm"], positions)
        k_cache.view(-1, case["kv_heads"], d)[where] = rotated(t["k"][at:at + n], t["k_norm"], positions)
        v_cache.view(-1, case["kv_heads"], d)[where] = t["v"][at:at + n].double()
        at += n
    return {"q": q_out, "k_cache": k_cache, "v_cache": v_cache}


def _exact_heads(q, k, v, limit):
    """One sequence in 64 bits, a head at a time; limit [n]: row i sees keys 0 .. limit[i] - 1."""
    n, hq, d = q.shape
    length, g = k.shape[0], hq // k.shape[1]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    if length == 0:
        return out, lse
    keys = torch.arange(length, device=q.device)
    rows = max(1, (1 << 28) // length)
    for h in range(hq):
        kh, vh = k[:, h // g].double(), v[:, h // g].double()
        for a in range(0, n, rows):
            s = (q[a:a + rows, h].double() @ kh.T) / math.sqrt(d)
            s.masked_fill_(keys[None, :] >= limit[a:a + rows, None], -math.inf)
            l = torch.logsumexp(s, dim=1)
            lse[h, a:a + rows] = l
            w = torch.exp(s - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None])
            out[a:a + rows, h] = w @ vh
    return out, lse


def _exact_paged(case, t):
    new, ctx = _lengths(case)
    dev = t["q"].device
    outs, lses, at = [], [], 0
    for s, (n, before) in enumerate(zip(new, ctx)):
        length = n + before
        keys = torch.arange(length, device=dev)
        where = t["table"][s].long()[keys // case["page"]] * case["page"] + keys % case["page"]
        k = t["k_cache"].view(-1, case["kv_heads"], case["d"])[where]
        v = t["v_cache"].view(-1, case["kv_heads"], case["d"])[where]
        limit = torch.full((n,), length, device=dev)
        if case["block"]:
            limit = torch.minimum(limit, (torch.arange(before, length, device=dev) // case["block"] + 1) * case["block"])
        o, l = _exact_heads(t["q"][at:at + n], k, v, limit)
        outs.append(o)
        lses.append(l)
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses, dim=1)}


def _exact_cross(case, t):
    outs, lses = [], []
    for b, length in enumerate(_key_lengths(case)):
        limit = torch.full((case["n"],), length, device=t["q"].device)
        o, l = _exact_heads(t["q"][b], t["k"][b], t["v"][b], limit)
        outs.append(o)
        lses.append(l)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
