"""Plain 64-bit forms of the 8-bit paged cache, of gathered attention weights and of eviction, with bounds that follow
from the kernels' arithmetic; shared by their tests."""
import math

import torch

from streaming_ref import Paged, attend, attention_bounds

BLOCK, E_MIN, E_MAX = 16, -15, 7
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


def powers(e):
    """2^e in 64 bits, exactly (e an integer tensor)."""
    return torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)[e.long() + 200]


def least_exponent(amax):
    """The least e in range with amax <= 448 * 2^e."""
    bounds = 448 * powers(torch.arange(E_MIN, E_MAX, device=amax.device))
    return E_MIN + (amax[..., None] > bounds).sum(-1)


def half_step8(x):
    """Half a step of e4m3 at |x| (codes: 2^-6 is its least normal number)."""
    low = torch.bucketize(x.abs(), powers(torch.arange(-5, 9, device=x.device)), right=True) - 6
    return powers(low - 4)


def round8(x):
    """To e4m3, nearest even, clamped, in 64 bits."""
    step = 2 * half_step8(x)
    return (torch.round(x / step) * step).clamp(-448, 448)


def codes64(c):
    return c.view(torch.uint8).view(CODE).float().double()


def exps(s):
    return s.view(torch.uint8).int() - 127


class Paged8:
    """A random 8-bit paged cache with its sequences; slots that no sequence owns hold NaN codes and scales."""

    def __init__(self, d, Hkv, page, lens, seed, order="token", spare=3, width=None, gain=1.0, scale_order="head"):
        base = Paged(torch.bfloat16, d, Hkv, page, lens, seed, order="token", spare=spare, width=width)
        self.lens, self.page, self.d, self.Hkv, self.table, self.kv_len = lens, page, d, Hkv, base.table, base.kv_len
        dev, total = base.k.device, base.k.shape[0]
        blocks = -(-page // BLOCK)

        def pool():
            shape = (total, page, Hkv, d) if order == "token" else (total, Hkv, page, d)
            c = torch.full(shape, 0x7f, dtype=torch.uint8, device=dev).view(CODE)
            c = c if order == "token" else c.transpose(1, 2)
            s = torch.full((total, blocks, Hkv) if scale_order == "head" else (Hkv, total, blocks), 0xff, dtype=torch.uint8, device=dev)
            s = s.view(SCALE)
            return c, s if scale_order == "head" else s.permute(1, 2, 0)
        (self.k, self.k_scale), (self.v, self.v_scale) = pool(), pool()
        g = torch.Generator(device=dev).manual_seed(seed + 1)
        # heads and stretches of tokens of very different size: scales differ from block to block
        for s, n in enumerate(lens):
            size = gain * torch.exp2(torch.randint(-6, 4, (n // 11 + 1, Hkv, 1), generator=g, device=dev).float())
            size = size.repeat_interleave(11, dim=0)[:n]
            for c, sc in ((self.k, self.k_scale), (self.v, self.v_scale)):
                self.put(c, sc, s, 0, (torch.randn(n, Hkv, d, generator=g, device=dev) * size).double())

    def cache(self, vdx):
        return vdx.PagedKV(self.k, self.v, self.table, self.k_scale, self.v_scale)

    def spots(self, s, first, n):
        c = torch.arange(first, first + n, device=self.table.device)
        return self.table[s].long()[c // self.page], c % self.page

    def put(self, codes, scales, s, first, x):
        """Tokens first, first + 1, .. of sequence s with values x [n, Hkv, d] (64 bits), by the definition."""
        bits, sc = codes.view(torch.uint8), scales.view(torch.uint8)
        a, end = first, first + x.shape[0]
        while a < end:
            page, slot = int(self.table[s, a // self.page]), a % self.page
            b = slot // BLOCK
            stop = min(end, a - slot + min(self.page, (b + 1) * BLOCK))
            e = least_exponent(x[a - first:stop - first].abs().amax((0, 2)))
            if slot > b * BLOCK:
                before = (sc[page, b].int() - 127).clamp(E_MIN, E_MAX)
                e = torch.maximum(e, before)
                old = bits[page, b * BLOCK:slot].view(CODE).float().double() * powers(before - e)[None, :, None]
                bits[page, b * BLOCK:slot] = round8(old).float().to(CODE).view(torch.uint8)
            bits[page, slot:slot + stop - a] = round8(x[a - first:stop - first] * powers(-e)[None, :, None]).float().to(CODE).view(torch.uint8)
            sc[page, b] = (e + 127).to(torch.uint8)
            a = stop

    def get(self, codes, scales, s, n=None):
        """Values of the first n tokens of sequence s in 64 bits."""
        page, slot = self.spots(s, 0, self.lens[s] if n is None else n)
        e = (scales.view(torch.uint8)[page, slot // BLOCK].int() - 127).clamp(E_MIN, E_MAX)
        return codes.view(torch.uint8)[page, slot].view(CODE).float().double() * powers(e)[..., None]

    def clone(self):
        other = object.__new__(type(self))
        other.__dict__.update(self.__dict__)
        for n in ("k", "v", "k_scale", "v_scale"):
            setattr(other, n, getattr(self, n).view(torch.uint8).clone().view(getattr(self, n).dtype))
        return other


def check_attention8(got_out, got_lse, ref, dtype, name=""):
    """As streaming_ref.check_attention, with what weights lose in fp16 where a kernel rounds them to it whatever the
    type: half of 2^-24 against a largest weight of at least 2^7, 2^-32 of it for each key."""
    o, lse, A, V, smax = ref
    bo, bl = attention_bounds(o, lse, A, V, smax, dtype)
    bo = bo + 2.0 ** -32 * (V[None] + 1)
    err = (got_out.double() - o).abs()
    assert bool((err <= bo).all()), (name, "out", float((err / bo.clamp_min(1e-300)).max()), float(err.max()))
    empty = torch.isinf(lse)
    assert bool((got_lse[empty] == -math.inf).all()), (name, "lse of rows without keys")
    le = (got_lse.double() - lse)[~empty].abs()
    assert bool((le <= bl[~empty]).all()), (name, "lse", float((le / bl[~empty]).max()) if le.numel() else 0)


def weigh(q, k, limit, lse, scale=None):
    """One sequence: q [n, Hq, d], k [L, Hkv, d], limit [n], lse [Hq, n] -> gathered weights [Hkv, L] in 64 bits and the
    error that fp32 work may make in each.  A score is an fp32 sum of d exact products (at most d * 2^-23 of their absolute
    sum), scaled (three roundings) and taken from lse (rounded to log2 units, and the difference); the exponential
    is within 2^-21; a key's sum over R rows loses at most R * 2^-23."""
    n, Hq, d = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    g = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    w = torch.zeros((Hkv, L), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(w)
    keys = torch.arange(L, device=q.device)
    for h in range(Hq):
        qq, kk = q[:, h].double(), k[:, h // g].double()
        s = (qq @ kk.T) * scale
        s = s.masked_fill(keys[None] >= limit[:, None], -math.inf)
        l = lse[h].double()
        s = torch.where(torch.isinf(l)[:, None], torch.full_like(s, -math.inf), s)
        l = torch.where(torch.isinf(l), torch.zeros_like(l), l)
        p = torch.exp(s - l[:, None])
        size = (qq.abs() @ kk.abs().T) * abs(scale)
        w[h // g] += p.sum(0)
        bound[h // g] += (p * ((d + 8) * 2.0 ** -23 * size + 2.0 ** -22 * l.abs()[:, None] + 2.0 ** -21 + n * g * 2.0 ** -23)).sum(0)
    return w, bound + 2.0 ** -126 * n * g


def stay(w, length, keep, recent):
    """Which of the keys of one head stay (indices in order), by sorting."""
    if length <= keep:
        return list(range(length))
    w = w[:length].tolist()
    def rank(i):
        return (-math.inf if math.isnan(w[i]) else 0, 0 if math.isnan(w[i]) else -w[i], i)
    older = sorted(range(length - recent), key=rank)[:keep - recent]
    return sorted(older) + list(range(length - recent, length))


__all__ = ["attend"]
