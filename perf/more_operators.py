"""Measured cases of the operators that keep a streaming cache small: appending to a paged key/value cache that is held
in 8 bits with a scale for each block of 16 tokens and head, attention over such a cache, the attention weight
that each cached key gathers, and the eviction of the keys that gathered least.

Head counts, head dimensions, grids, rotary sections and theta are those of the Wan-shaped workloads in
video_diffusion_transformer_rope_gb300/configs.py (12 and 40 heads of 128, 30x52 and 45x80 latent frames, 21 of
them; the tiny one has 4 heads of 64).

The cache: a block is 16 tokens of a page (the last one of a page may be short); its scale for a head is 2^e, the
least with |x| <= 448 * 2^e for all its values, e in [-15, 7] (held as float8_e8m0fnu); values are x * 2^-e rounded to
float8_e4m3fn.  New tokens that join older ones in a block can raise its scale: the older values are rounded again.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
SECTIONS = {128: (44, 42, 42), 64: (24, 20, 20)}
THETA = 10000.0
EPS = 1e-6
BLOCK = 16
E_MIN, E_MAX = -15, 7
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------------------------------------ cases
def _append(name, **kw):
    return dict(dict(name=name, op="append", dtype="bf16", d=128, seqs=1, heads=12, kv_heads=12, new_min=1, new_max=1,
                     ctx_min=0, ctx_max=0, page=128, frames=1024, rows=30, cols=52, norm=True, offset=0, layout=1), **kw)


def _attend(name, **kw):
    return dict(dict(name=name, op="attend", dtype="bf16", d=128, seqs=1, heads=12, kv_heads=12, new_min=1, new_max=1,
                     ctx_min=0, ctx_max=0, page=128, block=0, layout=1), **kw)


def _weigh(name, **kw):
    return dict(dict(name=name, op="weigh", dtype="bf16", bits=8, d=128, seqs=1, heads=12, kv_heads=12, new_min=1, new_max=1,
                     ctx_min=0, ctx_max=0, page=128, block=0, decay=1.0, layout=1), **kw)


def _evict(name, **kw):
    return dict(dict(name=name, op="evict", dtype="bf16", bits=8, d=128, seqs=1, kv_heads=12, len_min=1, len_max=1, page=128,
                     keep=1, recent=0, layout=1), **kw)


def listed():
    return [
        # one new token for each of eight sequences, most of them inside a block: the smallest append, all latency
        _append("append_token", seqs=8, ctx_min=100, ctx_max=2000, page=16, rows=1, cols=1, frames=4096),
        # three 720p latent frames for a guided pair behind one: the largest append, all bandwidth
        _append("append_chunk_720p", seqs=2, heads=40, kv_heads=40, new_min=10800, new_max=10800, ctx_min=3600, ctx_max=3600,
                page=128, rows=45, cols=80),
        # ragged prompts with grouped heads, half precision, no norm, chunks that begin and end inside blocks
        _append("append_ragged_fp16", dtype="fp16", d=64, seqs=13, kv_heads=4, new_min=1, new_max=301, ctx_min=0, ctx_max=500,
                page=32, norm=False, rows=1, cols=1, frames=4096),
        # a few sequences at one token each over short caches: latency
        _attend("attend_token_small", seqs=4, ctx_min=64, ctx_max=1000, page=16),
        # many sequences at one token each over long caches with grouped heads: reading the cache
        _attend("attend_token_large", seqs=48, heads=40, kv_heads=8, ctx_min=8000, ctx_max=32759, page=64),
        # a 720p latent frame over 21 frames: the largest chunk, all products
        _attend("attend_frame_720p", heads=40, kv_heads=40, new_min=3600, new_max=3600, ctx_min=72000, ctx_max=72000, page=128,
                block=3600),
        # ragged chunks, every token after the ones before it, grouped heads, half precision
        _attend("attend_ragged_fp16", dtype="fp16", d=64, seqs=9, kv_heads=4, new_min=1, new_max=500, ctx_min=0, ctx_max=3000,
                page=16, block=1),
        # what the single tokens of many sequences weighed, added up at every step: reading the keys
        _weigh("weigh_token", seqs=48, heads=40, kv_heads=8, ctx_min=8000, ctx_max=32759, page=64),
        # what a 480p latent frame weighed over 21 frames of a 16-bit cache, a page per frame, both halves of a guided pair
        _weigh("weigh_frame_480p", bits=16, seqs=2, new_min=1560, new_max=1560, ctx_min=31200, ctx_max=31200, page=1560, block=1560),
        # ragged chunks, grouped heads, half precision, older weights fading
        _weigh("weigh_ragged_fp16", dtype="fp16", d=64, seqs=9, kv_heads=4, new_min=1, new_max=500, ctx_min=0, ctx_max=3000,
               page=16, block=1, decay=0.9),
        # four short sequences cut down to 500 tokens, a few of them not yet that long: latency
        _evict("evict_small", seqs=4, len_min=300, len_max=2000, page=16, keep=500, recent=64),
        # 21 frames of 720p cut down to eight, the last one whole, 16 bits: the largest, all bandwidth
        _evict("evict_720p", bits=16, kv_heads=40, len_min=75600, len_max=75600, page=128, keep=28800, recent=3600),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_once(rng):
    heads, kv = rng.choice([(12, 12), (40, 40), (12, 4), (40, 8), (4, 4), (40, 40), (12, 12), (12, 1)])
    common = dict(dtype=rng.choice(["bf16", "bf16", "fp16"]), d=rng.choice([128, 128, 64]), kv_heads=kv, layout=rng.randrange(1 << 30))
    op = rng.choice(["append", "attend", "weigh", "evict"])
    page = rng.choice([16, 32, 64, 128, 200, 1560, 3600])
    bits = rng.choice([8, 8, 16])
    if op == "evict":
        top = _log(rng, 1, 75600)
        keep = _log(rng, 1, 30000)
        return _evict("", bits=bits, seqs=_log(rng, 1, 64), len_min=rng.choice([0, top // 2, top]), len_max=top, page=page, keep=keep,
                      recent=rng.choice([0, keep // 8, keep // 2, keep]), **common)
    new = _log(rng, 1, 10800 if op == "append" else 3600)
    ctx = _log(rng, 1, 4000 if op == "append" else 72000)
    ranges = dict(seqs=_log(rng, 1, 64), new_min=rng.choice([1, max(1, new // 2), new]), new_max=new,
                  ctx_min=rng.choice([0, ctx // 2, ctx]), ctx_max=ctx, page=page, heads=heads)
    if op == "append":
        rows, cols, frames = rng.choice([(30, 52, 1024), (45, 80, 1024), (1, 1, 32768)])
        return _append("", rows=rows, cols=cols, frames=frames, norm=rng.random() < 0.5, offset=rng.choice([0, 0, 1560, 14400]),
                       **ranges, **common)
    block = rng.choice([0, 1, 1560, 3600])
    if op == "attend":
        return _attend("", block=block, **ranges, **common)
    return _weigh("", bits=bits, block=block, decay=rng.choice([1.0, 0.9]), **ranges, **common)


_CAP = {}


def draw(rng):
    if not _CAP:
        for c in listed():
            w, cap = work(c), _CAP.setdefault(c["op"], {"bytes": 0, "flops": 0, "held": 0, "padded": 0})
            for what, n in (("bytes", w["bytes"]), ("flops", w["flops"]), ("held", _held(c)), ("padded", _padded(c))):
                cap[what] = max(cap[what], n)
    while True:
        c = _draw_once(rng)
        w, cap = work(c), _CAP[c["op"]]
        if w["bytes"] <= cap["bytes"] and w["flops"] <= cap["flops"] and _held(c) <= cap["held"] and _padded(c) <= 4 * cap["padded"]:
            del c["name"]
            return c


# ------------------------------------------------------------------------------------------------ shapes
def _lengths(case):
    """New tokens and cached tokens before them, for each sequence: part of the case, not of the seed."""
    r = random.Random(case["layout"])
    if case["op"] == "evict":
        return [0] * case["seqs"], [r.randint(case["len_min"], case["len_max"]) for _ in range(case["seqs"])]
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["seqs"])]
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    return new, ctx


def _key_bytes(case):
    """Bytes of one key or value of one head, its share of a block's scale with it."""
    return case["d"] + 1 / BLOCK if case.get("bits", 8) == 8 else 2 * case["d"]


def _held(case):
    """Bytes of the caches that a case keeps."""
    new, ctx = _lengths(case)
    pages = sum(-(-(a + b) // case["page"]) for a, b in zip(new, ctx))
    if case["op"] == "evict":
        pages += sum(-(-min(n, case["keep"]) // case["page"]) for n in ctx)
    return 2 * pages * case["page"] * case["kv_heads"] * _key_bytes(case)


def _padded(case):
    """Elements of the keys and scores of all sequences, each as long as the longest: what a plain form holds at once."""
    new, ctx = _lengths(case)
    if case["op"] == "append":
        return sum(new)
    group = 1 if case["op"] == "evict" else case["heads"] // case["kv_heads"]
    return case["seqs"] * case["kv_heads"] * max(a + b for a, b in zip(new, ctx)) * (max(new) * group + case["d"])


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
    hk, d = case["kv_heads"], case["d"]
    new, ctx = _lengths(case)
    key = _key_bytes(case)
    if case["op"] == "evict":
        kept = [min(n, case["keep"]) for n in ctx]
        return {"bytes": int(4 * hk * sum(ctx) + (4 * key + 4 + 4) * hk * sum(kept)), "flops": 0}
    hq, n = case["heads"], sum(new)
    if case["op"] == "append":
        return {"bytes": int(2 * n * (2 * hq + 2 * hk) * d + 2 * n * hk * key), "flops": (10 if case["norm"] else 6) * n * (hq + hk) * d}
    pairs = sum(_visible(a, a + b, case["block"]) for a, b in zip(new, ctx))
    keys = sum(a + b for a, b in zip(new, ctx))
    if case["op"] == "attend":
        return {"bytes": int(4 * n * hq * d + 4 * n * hq + 2 * keys * hk * key), "flops": 4 * d * hq * pairs}
    return {"bytes": int(2 * n * hq * d + 4 * n * hq + keys * hk * key + 4 * hk * (keys + sum(ctx))), "flops": 2 * d * hq * pairs}


# ------------------------------------------------------------------------------------------------ 8-bit blocks
def _two_to(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e in its range with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    return torch.where(m <= 0.875, x - 9, x - 8).clamp(E_MIN, E_MAX).to(torch.int32)


def _round8(x):
    return x.clamp(-448.0, 448.0).to(CODE)


def _store8(codes, scales, values, page, slot, seq_first):
    """Write tokens of 32-bit values [n, heads, d] to slots of pages: codes [pages, P, heads, d], scales [pages, blocks, heads].
    seq_first: (page, slot) of each sequence's first new token; the tokens ahead of it in its block are older ones."""
    pages, P, heads, d = codes.shape
    blocks = scales.shape[1]
    bits, exps = codes.view(torch.uint8), scales.view(torch.uint8).view(pages * blocks, heads)
    b = page * blocks + slot // BLOCK
    amax = torch.zeros((pages * blocks, heads), dtype=torch.float32, device=values.device)
    amax.index_reduce_(0, b, values.abs().amax(dim=-1), "amax")
    e = _exponent(amax)
    if seq_first is not None:
        page0, slot0 = seq_first
        inside = slot0 % BLOCK > 0
        page0, slot0 = page0[inside], slot0[inside]
        b0 = page0 * blocks + slot0 // BLOCK
        before = exps[b0].to(torch.int32) - 127
        e[b0] = torch.maximum(e[b0], before)
        at = (slot0 // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device=slot0.device)[None, :]
        older = at < slot0[:, None]
        which = older.nonzero()[:, 0]
        pg, sl = page0[which], at[older]
        value = bits[pg, sl].view(CODE).float() * _two_to(before - e[b0])[which][..., None]
        bits[pg, sl] = _round8(value).view(torch.uint8)
    exps[b] = (e[b] + 127).to(torch.uint8)
    bits[page, slot] = _round8(values * _two_to(-e[b])[..., None]).view(torch.uint8)


def _load8(codes, scales, page, slot):
    """The values of slots (any shape of page and slot) in 32 bits: [..., heads, d]."""
    e = scales.view(torch.uint8)[page, slot // BLOCK].to(torch.int32) - 127
    return codes.view(torch.uint8)[page, slot].view(CODE).float() * _two_to(e)[..., None]


# ------------------------------------------------------------------------------------------------ inputs
def _table(pages, total, order, dev):
    """Pages of each sequence, dealt out in `order`."""
    owner = torch.repeat_interleave(torch.arange(len(pages), device=dev), torch.tensor(pages, device=dev), output_size=total)
    start = torch.tensor([sum(pages[:s]) for s in range(len(pages))], device=dev)
    table = torch.zeros((len(pages), max(1, max(pages))), dtype=torch.int32, device=dev)
    table[owner, torch.arange(total, device=dev) - start[owner]] = order[:total]
    return table


def prepare(case, seed):
    """Tensors of a case, from the seed alone: activations of about unit variance with a few strong channels (as
    projections give them), heads of different gains, queries that make attention moderately peaked."""
    dev, dt = torch.device("cuda"), DT[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 29)
    hk, d, P = case["kv_heads"], case["d"], case["page"]
    new, ctx = _lengths(case)
    length = [a + b for a, b in zip(new, ctx)]
    eight = case.get("bits", 8) == 8
    gain = torch.exp2(torch.randint(-2, 3, (hk, 1), generator=g, device=dev).float())

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def pool(pages, fill):
        shape, step = (max(1, pages), P, hk, d), max(1, 65536 // P)
        if not eight:
            c = torch.zeros(shape, dtype=dt, device=dev)
            for i in range(0, pages if fill else 0, step):
                c[i:i + step] = (randn(*c[i:i + step].shape) * gain).to(dt)
            return c, None
        c = torch.zeros(shape, dtype=CODE, device=dev)
        s = torch.full((max(1, pages), -(-P // BLOCK), hk), 127, dtype=torch.uint8, device=dev).view(SCALE)
        for i in range(0, pages if fill else 0, step):
            n = min(step, pages - i)
            page, slot = torch.arange(n, device=dev).repeat_interleave(P), torch.arange(P, device=dev).repeat(n)
            _store8(c[i:i + n], s[i:i + n], randn(n * P, hk, d) * gain, page, slot, None)
        return c, s

    pages = [-(-n // P) for n in length]
    total = sum(pages)
    t = {"table": _table(pages, total, torch.randperm(max(1, total), generator=g, device=dev).to(torch.int32), dev)}
    t["k_cache"], t["k_scale"] = pool(total, True)
    t["v_cache"], t["v_scale"] = pool(total, case["op"] != "weigh")
    t["kv_len"] = torch.tensor(length, dtype=torch.int32, device=dev)
    t["cu"] = torch.tensor([sum(new[:s]) for s in range(len(new) + 1)], dtype=torch.int32, device=dev)
    n = sum(new)
    if case["op"] == "append":
        hq = case["heads"]
        qkv = torch.empty((n, hq + 2 * hk, d), dtype=dt, device=dev)      # one projection's output, side by side
        for i in range(0, n, 4096):
            qkv[i:i + 4096] = randn(*qkv[i:i + 4096].shape).to(dt)
        qkv[:, :, d // 3] *= 4
        t["q"], t["k"], t["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        t["offset"] = torch.full((case["seqs"],), case["offset"], dtype=torch.int32, device=dev) if case["offset"] else None
        t["q_norm"] = (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None
        t["k_norm"] = (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None
    elif case["op"] == "evict":
        # weights as long generation leaves them: a few heavy keys, many light ones, some never looked at
        w = torch.exp(2 * randn(case["seqs"], hk, max(1, max(length))))
        t["weights"] = w.masked_fill_(randn(*w.shape) > 1.5, 0.0)
        kept = [-(-min(m, case["keep"]) // P) for m in length]
        t["into_table"] = _table(kept, sum(kept), torch.randperm(max(1, sum(kept)), generator=g, device=dev).to(torch.int32), dev)
        t["into_k"], t["into_k_scale"] = pool(sum(kept), False)
        t["into_v"], t["into_v_scale"] = pool(sum(kept), False)
        t["offset"] = torch.arange(case["seqs"], dtype=torch.int32, device=dev)
    else:
        q = randn(n, case["heads"], d) * 1.5 / gain.repeat_interleave(case["heads"] // hk, dim=0)
        t["q"] = q.to(dt)
    st = {"case": case, "t": t, "new": new, "len": length}
    if case["op"] == "weigh":
        t["lse"] = _plain_lse(st)
        t["weights"] = torch.rand((case["seqs"], hk, max(length)), generator=g, device=dev)
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "weigh": _own_weigh, "evict": _own_evict}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}[op](state)


def _own_append(st):
    import video_diffusion_transformer_rope_gb300 as vdx
    c, t = st["case"], st["t"]
    cache = vdx.PagedKV(t["k_cache"], t["v_cache"], t["table"], t["k_scale"], t["v_scale"])
    q = vdx.rope3d_append(t["q"], t["k"], t["v"], cache, t["cu"], t["kv_len"], (c["frames"], c["rows"], c["cols"]),
                          sections=SECTIONS[c["d"]], theta=THETA, pos_offset=t["offset"], q_norm=t["q_norm"],
                          k_norm=t["k_norm"], eps=EPS)
    return {"q": q, "k_cache": t["k_cache"], "k_scale": t["k_scale"], "v_cache": t["v_cache"], "v_scale": t["v_scale"]}


def _own_attend(st):
    import video_diffusion_transformer_rope_gb300 as vdx
    c, t = st["case"], st["t"]
    cache = vdx.PagedKV(t["k_cache"], t["v_cache"], t["table"], t["k_scale"], t["v_scale"])
    out, lse = vdx.paged_attn(t["q"], cache, t["cu"], t["kv_len"], max_q=max(st["new"]), max_kv=max(st["len"]),
                              causal_block=c["block"])
    return {"out": out, "lse": lse}


def _own_weigh(st):
    import video_diffusion_transformer_rope_gb300 as vdx
    c, t = st["case"], st["t"]
    cache = vdx.PagedKV(t["k_cache"], t["v_cache"], t["table"], t["k_scale"], t["v_scale"])
    vdx.paged_attn_weights(t["q"], cache, t["cu"], t["kv_len"], t["lse"], t["weights"], max_q=max(st["new"]), max_kv=max(st["len"]),
                           causal_block=c["block"], decay=c["decay"])
    return {"weights": t["weights"]}


def _own_evict(st):
    import video_diffusion_transformer_rope_gb300 as vdx
    c, t = st["case"], st["t"]
    cache = vdx.PagedKV(t["k_cache"], t["v_cache"], t["table"], t["k_scale"], t["v_scale"])
    into = vdx.PagedKV(t["into_k"], t["into_v"], t["into_table"], t["into_k_scale"], t["into_v_scale"])
    left = vdx.paged_evict(cache, t["weights"], t["kv_len"], c["keep"], into, recent=c["recent"], max_kv=max(1, max(st["len"])),
                           pos_offset=t["offset"])
    return _evicted(t, left.kv_len, left.pos_offset, left.weights, left.index)


def _evicted(t, kv_len, offset, weights, index):
    out = {"kv_len": kv_len, "pos_offset": offset, "weights": weights, "index": index, "k": t["into_k"], "v": t["into_v"]}
    if t["into_k_scale"] is not None:
        out.update(k_scale=t["into_k_scale"], v_scale=t["into_v_scale"])
    return out


def _plain_append(st):
    c, t = st["case"], st["t"]
    dev, d, n = t["q"].device, c["d"], t["q"].shape[0]
    count = (t["cu"][1:] - t["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device=dev), count, output_size=n)
    first = t["kv_len"].long() - count                    # cache index of each sequence's first new token
    index = first[seq] + torch.arange(n, device=dev) - t["cu"].long()[seq]
    pos = index + (t["offset"].long()[seq] if t["offset"] is not None else 0)
    area = c["rows"] * c["cols"]
    st_, sh, sw = SECTIONS[d]

    def angles(coord, section):
        return coord.double()[:, None] * THETA ** (-2.0 * torch.arange(section // 2, device=dev, dtype=torch.float64) / section)

    angle = torch.cat([angles(pos // area, st_), angles(pos // c["cols"] % c["rows"], sh), angles(pos % c["cols"], sw)], dim=1)
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()
        even, odd = x[..., 0::2], x[..., 1::2]
        y = torch.empty_like(x)
        y[..., 0::2] = even * cos - odd * sin
        y[..., 1::2] = even * sin + odd * cos
        return y

    P, seqs = c["page"], torch.arange(c["seqs"], device=dev)
    page, slot = t["table"].long()[seq, index // P], index % P
    seq_first = t["table"].long()[seqs, first // P], first % P
    _store8(t["k_cache"], t["k_scale"], turn(t["k"], t["k_norm"]), page, slot, seq_first)
    _store8(t["v_cache"], t["v_scale"], t["v"].float(), page, slot, seq_first)
    return {"q": turn(t["q"], t["q_norm"]).to(t["q"].dtype), "k_cache": t["k_cache"], "k_scale": t["k_scale"],
            "v_cache": t["v_cache"], "v_scale": t["v_scale"]}


def _padded_scores(st, use, budget=1 << 30):
    """Scores of all sequences side by side, padded, some kv heads at a time, in 32 bits: use(a, b, scores [seqs, b - a,
    group * rows, keys] with -inf where a row sees no key, gather) with gather(codes, scales) those heads of a cache."""
    c, t = st["case"], st["t"]
    dev, hk, g, d, P, S = t["q"].device, c["kv_heads"], c["heads"] // c["kv_heads"], c["d"], c["page"], c["seqs"]
    n, length = max(st["new"]), max(st["len"])
    rows = torch.arange(n, device=dev)
    keys = torch.arange(length, device=dev)
    count = (t["cu"][1:] - t["cu"][:-1]).long()
    at = t["cu"][:-1].long()[:, None] + rows[None, :]
    live = rows[None, :] < count[:, None]
    q = t["q"][at.clamp(max=t["q"].shape[0] - 1)]                         # [seqs, rows, Hq, d]
    kv_len = t["kv_len"].long()
    p = (kv_len - count)[:, None] + rows[None, :]
    limit = kv_len[:, None].expand(S, n) if c["block"] == 0 else torch.minimum((p // c["block"] + 1) * c["block"], kv_len[:, None])
    seen = (keys[None, None, :] < limit[:, :, None]) & live[:, :, None]   # [seqs, rows, keys]
    page, slot = t["table"].long()[:, keys // P], keys % P
    step = max(1, budget // (S * length * (g * n + 2 * d)))
    for a in range(0, hk, step):
        b = min(hk, a + step)

        def gather(cache, scale):
            if scale is None:
                return cache[:, :, a:b][page, slot].float().transpose(1, 2)
            return _load8(cache[:, :, a:b], scale[:, :, a:b], page, slot.expand_as(page)).transpose(1, 2)

        qh = q[:, :, a * g:b * g].float().view(S, n, b - a, g, d).permute(0, 2, 3, 1, 4).reshape(S, b - a, g * n, d)
        s = torch.matmul(qh, gather(t["k_cache"], t["k_scale"]).transpose(2, 3)) * d ** -0.5
        s = s.view(S, b - a, g, n, length).masked_fill_(~seen[:, None, None], -math.inf).view(S, b - a, g * n, length)
        use(a, b, s, gather)
    return live


def _plain_attend(st):
    c, t = st["case"], st["t"]
    S, hq, g, n, d = c["seqs"], c["heads"], c["heads"] // c["kv_heads"], max(st["new"]), c["d"]
    out = torch.zeros((S, n, hq, d), dtype=t["q"].dtype, device=t["q"].device)
    lse = torch.zeros((S, n, hq), dtype=torch.float32, device=out.device)

    def use(a, b, s, gather):
        m = s.amax(dim=-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        total = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p, gather(t["v_cache"], t["v_scale"])) / torch.where(total == 0, torch.ones_like(total), total)
        out[:, :, a * g:b * g] = o.view(S, b - a, g, n, d).permute(0, 3, 1, 2, 4).reshape(S, n, (b - a) * g, d).to(out.dtype)
        lse[:, :, a * g:b * g] = (m + torch.log(total)).view(S, b - a, g, n).permute(0, 3, 1, 2).reshape(S, n, (b - a) * g)

    live = _padded_scores(st, use)
    return {"out": out[live], "lse": lse[live].t().contiguous()}


def _plain_lse(st):
    c, t = st["case"], st["t"]
    S, hq, g, n = c["seqs"], c["heads"], c["heads"] // c["kv_heads"], max(st["new"])
    lse = torch.zeros((S, n, hq), dtype=torch.float32, device=t["q"].device)

    def use(a, b, s, gather):
        lse[:, :, a * g:b * g] = torch.logsumexp(s, dim=-1).view(S, b - a, g, n).permute(0, 3, 1, 2).reshape(S, n, (b - a) * g)

    return lse[_padded_scores(st, use)].t().contiguous()


def _plain_weigh(st):
    c, t = st["case"], st["t"]
    S, g, n, length = c["seqs"], c["heads"] // c["kv_heads"], max(st["new"]), max(st["len"])
    dev = t["q"].device
    count = (t["cu"][1:] - t["cu"][:-1]).long()
    keys = torch.arange(length, device=dev)
    rows = (t["cu"][:-1].long()[:, None] + torch.arange(n, device=dev)[None, :]).clamp(max=t["q"].shape[0] - 1)
    lse = t["lse"].t()[rows]                                              # [seqs, rows, Hq]
    kv_len = t["kv_len"].long()
    older = keys[None, :] < (kv_len - count)[:, None]
    old = torch.where(older[:, None], t["weights"] * c["decay"], torch.zeros_like(t["weights"]))

    def use(a, b, s, gather):
        l = lse[:, :, a * g:b * g].view(S, n, b - a, g).permute(0, 2, 3, 1).reshape(S, b - a, g * n, 1)
        old[:, a:b] += torch.exp(s - l).sum(dim=2)

    _padded_scores(st, use)
    held = (keys[None, :] < kv_len[:, None]) & (count > 0)[:, None]
    t["weights"].copy_(torch.where(held[:, None], old, t["weights"]))
    return {"weights": t["weights"]}


def _plain_evict(st):
    c, t = st["case"], st["t"]
    dev, hk, d, P, S, keep = t["weights"].device, c["kv_heads"], c["d"], c["page"], c["seqs"], c["keep"]
    width = t["weights"].shape[2]
    L = t["kv_len"].long()
    keys = torch.arange(width, device=dev)
    left = L.clamp(max=keep)
    order = t["weights"].masked_fill((keys[None, :] >= (L - c["recent"])[:, None])[:, None], math.inf)
    order = order.masked_fill((keys[None, :] >= L[:, None])[:, None], -math.inf)
    # the heaviest first, the lowest index among equals; behind the last key that stays, a number past all of them
    chosen = torch.sort(order, dim=-1, descending=True, stable=True).indices[..., :keep]
    j = torch.arange(chosen.shape[-1], device=dev)
    stays = (j[None, :] < left[:, None])[:, None]
    chosen = torch.sort(torch.where(stays, chosen, width), dim=-1).values
    index = torch.full((S, hk, keep), -1, dtype=torch.int32, device=dev)
    index[..., :chosen.shape[-1]] = torch.where(stays, chosen, -1)
    weights = torch.zeros((S, hk, keep), dtype=torch.float32, device=dev)
    weights[..., :chosen.shape[-1]] = torch.where(stays, t["weights"].gather(2, chosen.clamp(max=width - 1)), 0.0)

    seq, to = stays[:, 0].nonzero(as_tuple=True)                          # every token that stays: its sequence and new index
    src = chosen[seq, :, to]                                              # [tokens, heads]
    head = torch.arange(hk, device=dev)[None, :]
    page, slot = t["table"].long()[seq[:, None], src // P], src % P
    into = t["into_table"].long()[seq, to // P], to % P

    def move(cache, scale, into_cache, into_scale):
        if scale is None:
            into_cache[into] = cache[page, slot, head]
            return
        e = scale.view(torch.uint8)[page, slot // BLOCK, head].to(torch.int32) - 127
        value = cache.view(torch.uint8)[page, slot, head].view(CODE).float() * _two_to(e)[..., None]
        _store8(into_cache, into_scale, value, *into, None)

    move(t["k_cache"], t["k_scale"], t["into_k"], t["into_k_scale"])
    move(t["v_cache"], t["v_scale"], t["into_v"], t["into_v_scale"])
    return _evicted(t, left.to(torch.int32), (t["offset"] + L - left).to(torch.int32), weights, index)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 4e11 or _held(case) > 4e9:
        return None
    t = prepare(case, seed)["t"]
    return {"append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](case, t)


def _exact_block(values, older, older_scale):
    """One block of one cache: values [tokens, heads, d] of its new tokens behind `older` [tokens, heads, d] whose scales
    were older_scale [heads]; gives the block's codes and scales."""
    powers = _powers(E_MIN, E_MAX, values.device)
    need = (values.abs().amax(dim=(0, 2))[:, None] > 448 * powers[:-1]).sum(dim=1)
    scale = powers[need]
    if older.shape[0]:
        scale = torch.maximum(scale, older_scale)
    x = torch.cat([older, values]) / scale[None, :, None]
    step = _powers(-9, 5, x.device)[torch.bucketize(x.abs(), _powers(-5, 8, x.device), right=True)]
    return (torch.round(x / step) * step).clamp(-448, 448), scale


def _powers(a, b, device):
    return torch.tensor([2.0 ** e for e in range(a, b + 1)], dtype=torch.float64, device=device)


def _exact_store(codes, scales, values, table, first, P):
    """Tokens first, first + 1, ... of one sequence into 64-bit copies of its codes and scales (as powers of two)."""
    a, end = first, first + values.shape[0]
    while a < end:
        page, slot = int(table[a // P]), a % P
        top = slot // BLOCK * BLOCK
        stop = min(end, a - slot + min(P, top + BLOCK))
        scale = scales[page, slot // BLOCK]
        older = codes[page, top:slot] * scale[None, :, None]
        got, scale = _exact_block(values[a - first:stop - first], older, scale)
        codes[page, top:slot + stop - a] = got
        scales[page, slot // BLOCK] = scale
        a = stop


def _values(codes):
    return codes.float().double() if codes is not None else None


def _exact_append(case, t):
    d, P, dev = case["d"], case["page"], t["q"].device
    new, ctx = _lengths(case)
    if sum(new) * case["kv_heads"] > 60000:
        return None
    sections = SECTIONS[d]
    turns = torch.tensor([THETA ** (-2.0 * j / s) for s in sections for j in range(s // 2)], dtype=torch.float64, device=dev)

    def rotated(x, weight, positions):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + EPS) * weight.double()
        frame, rest = positions // (case["rows"] * case["cols"]), positions % (case["rows"] * case["cols"])
        coord = torch.stack([frame, rest // case["cols"], rest % case["cols"]], dim=1).double()
        coord = coord.repeat_interleave(torch.tensor([s // 2 for s in sections], device=dev), dim=1)
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous())
        z = z * torch.polar(torch.ones_like(coord), coord * turns)[:, None, :]
        return torch.view_as_real(z).reshape(x.shape)

    out = {"q": torch.empty(t["q"].shape, dtype=torch.float64, device=dev)}
    for name in ("k_cache", "k_scale", "v_cache", "v_scale"):
        out[name] = _values(t[name])
    at, table = 0, t["table"].tolist()
    for s, (n, before) in enumerate(zip(new, ctx)):
        positions = torch.arange(before, before + n, device=dev) + case["offset"]
        out["q"][at:at + n] = rotated(t["q"][at:at + n], t["q_norm"], positions)
        _exact_store(out["k_cache"], out["k_scale"], rotated(t["k"][at:at + n], t["k_norm"], positions), table[s], before, P)
        _exact_store(out["v_cache"], out["v_scale"], t["v"][at:at + n].double(), table[s], before, P)
        at += n
    return out


def _exact_keys(case, t, which, s, length):
    """Keys or values of one sequence in 64 bits, [length, heads, d]."""
    keys = torch.arange(length, device=t["table"].device)
    where = t["table"][s].long()[keys // case["page"]], keys % case["page"]
    x = _values(t[which + "_cache"].view(torch.uint8)[where].view(CODE)) if t[which + "_scale"] is not None else t[which + "_cache"][where].double()
    if t[which + "_scale"] is not None:
        x = x * _values(t[which + "_scale"].view(torch.uint8)[where[0], where[1] // BLOCK].view(SCALE))[..., None]
    return x


def _exact_rows(case, t):
    """Each sequence, head and run of rows: (sequence, head, first row, rows, scores in 64 bits with -inf where nothing is seen)."""
    new, ctx = _lengths(case)
    g, at = case["heads"] // case["kv_heads"], 0
    for s, (n, before) in enumerate(zip(new, ctx)):
        length = n + before
        k = _exact_keys(case, t, "k", s, length)
        limit = torch.full((n,), length, device=k.device)
        if case["block"]:
            limit = torch.minimum(limit, (torch.arange(before, length, device=k.device) // case["block"] + 1) * case["block"])
        step = max(1, (1 << 28) // max(1, length))
        for h in range(case["heads"]):
            for a in range(0, n, step):
                scores = t["q"][at + a:at + min(n, a + step), h].double() @ k[:, h // g].T / math.sqrt(case["d"])
                scores.masked_fill_(torch.arange(length, device=k.device)[None, :] >= limit[a:a + step, None], -math.inf)
                yield s, h, at + a, scores
        at += n


def _exact_attend(case, t):
    new, ctx = _lengths(case)
    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(t["q"].shape, dtype=torch.float64, device=t["q"].device)
    lse = torch.zeros((case["heads"], out.shape[0]), dtype=torch.float64, device=out.device)
    held = (-1, None)
    for s, h, a, scores in _exact_rows(case, t):
        if held[0] != s:
            held = s, _exact_keys(case, t, "v", s, new[s] + ctx[s])
        l = torch.logsumexp(scores, dim=1)
        lse[h, a:a + scores.shape[0]] = l
        out[a:a + scores.shape[0], h] = torch.exp(scores - l[:, None]) @ held[1][:, h // g]
    return {"out": out, "lse": lse}


def _exact_weigh(case, t):
    new, ctx = _lengths(case)
    g = case["heads"] // case["kv_heads"]
    w = t["weights"].double()
    for s, (n, before) in enumerate(zip(new, ctx)):
        w[s, :, :before] *= case["decay"]
        w[s, :, before:before + n] = 0
    for s, h, a, scores in _exact_rows(case, t):
        w[s, h // g, :scores.shape[1]] += torch.exp(scores - t["lse"][h, a:a + scores.shape[0]].double()[:, None]).sum(0)
    return {"weights": w}


def _exact_evict(case, t):
    new, ctx = _lengths(case)
    S, hk, P, keep = case["seqs"], case["kv_heads"], case["page"], case["keep"]
    weights = torch.zeros((S, hk, keep), dtype=torch.float64, device=t["weights"].device)
    caches = {n: _values(t["into_" + n]) if case["bits"] == 8 else t["into_" + n].double() for n in ("k", "v")}
    scales = {n: _values(t["into_" + n + "_scale"]) for n in ("k", "v")}
    into = t["into_table"].tolist()
    for s, length in enumerate(ctx):
        left = min(length, keep)
        chosen = []
        for h in range(hk):
            w = t["weights"][s, h, :length]
            if left < length:
                older = w[:length - min(case["recent"], keep)]
                need = keep - min(case["recent"], keep)
                border = torch.sort(older).values[older.shape[0] - need] if need else math.inf
                stays = older > border
                ties = (older == border).nonzero()[:, 0]
                stays[ties[:need - int(stays.sum())]] = True
                stays = torch.cat([stays, torch.ones(length - older.shape[0], dtype=torch.bool, device=w.device)])
            else:
                stays = torch.ones(length, dtype=torch.bool, device=w.device)
            chosen.append(stays.nonzero()[:, 0])
            weights[s, h, :left] = w[stays].double()
        if left == 0:
            continue
        for n in ("k", "v"):
            x = _exact_keys(case, t, n, s, length)
            x = torch.stack([x[chosen[h], h] for h in range(hk)], dim=1)
            if case["bits"] == 8:
                _exact_store(caches[n], scales[n], x, into[s], 0, P)
            else:
                where = torch.arange(left, device=x.device)
                caches[n][t["into_table"][s].long()[where // P], where % P] = x
    out = {"kv_len": None, "pos_offset": None, "weights": weights, "index": None, "k": caches["k"], "v": caches["v"]}
    if case["bits"] == 8:
        out.update(k_scale=scales["k"], v_scale=scales["v"])
    return out
