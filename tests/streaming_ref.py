"""Plain 64-bit forms of the paged-cache and cross-attention operations, and error bounds that
follow from the kernels' arithmetic; shared by the streaming tests."""
import math

import numpy as np
import torch

SECTIONS = {128: (44, 42, 42), 64: (24, 20, 20)}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rotate(x, pos, grid, sections, theta, weight=None, eps=0.0):
    """x [rows, H, d] (any float type), pos [rows] grid tokens -> [rows, H, d] float64."""
    x = x.double()
    d = x.shape[-1]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    _, Hg, Wg = grid
    parts = []
    for a, S in zip((pos // (Hg * Wg), pos // Wg % Hg, pos % Wg), sections):
        j = torch.arange(S // 2, dtype=torch.float64, device=x.device)
        parts.append(a.double()[:, None] * theta ** (-2.0 * j / S))
    ang = torch.cat(parts, dim=1)[:, None, :]
    c, s = torch.cos(ang), torch.sin(ang)
    y = torch.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    assert y.shape[-1] == d
    return y


def rotate_bound(ref, dtype):
    """One rounding to dtype (half a step of the value, or of the smallest normal number) plus fp32
    work: a pair's rotation and the norm's product chain stay within 32 units of 2^-24 of the pair's
    length (cos and sin within 2 ulp, three products, one fused sum, a sum of d squares)."""
    pair = torch.sqrt(ref[..., 0::2] ** 2 + ref[..., 1::2] ** 2).repeat_interleave(2, dim=-1)
    return half_step(dtype) * torch.maximum(ref.abs(), torch.full_like(ref, torch.finfo(dtype).tiny)) * 1.001 + 2.0 ** -19 * pair


def attend(q, k, v, limit, scale=None):
    """One sequence: q [n, Hq, d], k, v [L, Hkv, d], limit [n] -> out [n, Hq, d], lse [Hq, n], and what
    the bounds need: A = sum of weights * |v| [n, Hq, d], V = sum |v| over the keys [Hq, d], smax [Hq, n] = largest
    sum |q_i k_i| * scale of a row."""
    n, Hq, d = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((n, Hq, d), dtype=torch.float64, device=q.device)
    A = torch.zeros_like(out)
    V = torch.zeros((Hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64, device=q.device)
    smax = torch.zeros_like(lse)
    if n and L:
        keys = torch.arange(L, device=q.device)
        for h in range(Hq):
            kk, vv, qq = k[:, h // (Hq // Hkv)].double(), v[:, h // (Hq // Hkv)].double(), q[:, h].double()
            s = (qq @ kk.T) * scale
            s = s.masked_fill(keys[None] >= limit[:, None], -math.inf)
            m = s.amax(1, keepdim=True)
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            l = p.sum(1, keepdim=True)
            w = p / torch.where(l == 0, torch.ones_like(l), l)
            out[:, h], A[:, h] = w @ vv, w @ vv.abs()
            V[h] = vv.abs().sum(0)
            lse[h] = (m + torch.log(l))[:, 0]
            smax[h] = ((qq.abs() @ kk.abs().T) * abs(scale)).amax(1)
    return out, lse, A, V, smax


def attention_bounds(ref, lse, A, V, smax, dtype):
    """Weights are rounded to dtype (half a step each; below fp16's normal range half of 2^-24
    against a largest weight of at least 1), the output once; a score is an fp32 sum of d exact
    products (at most d * 2^-23 of their absolute sum, accumulated with truncation), used in log2
    units (two more roundings of the score and one of its distance to the running maximum), the
    exponential and the sums add 2^-19 in all."""
    d = ref.shape[-1]
    ds = (d + 8) * 2.0 ** -23 * smax + 2.0 ** -19
    rel = 2 * ds.T[..., None]
    u = half_step(dtype)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    out = u * 1.01 * (A + ref.abs()) + rel * A + tiny * (V[None] + 1)
    return out, ds + 2.0 ** -21 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).abs()


def check_attention(got_out, got_lse, ref, dtype, name=""):
    o, lse, A, V, smax = ref
    bo, bl = attention_bounds(o, lse, A, V, smax, dtype)
    err = (got_out.double() - o).abs()
    assert bool((err <= bo).all()), (name, "out", float((err / bo.clamp_min(1e-300)).max()), float(err.max()))
    empty = torch.isinf(lse)
    assert bool((got_lse[empty] == -math.inf).all()), (name, "lse of rows without keys")
    le = (got_lse.double() - lse)[~empty].abs()
    assert bool((le <= bl[~empty]).all()), (name, "lse", float((le / bl[~empty]).max()) if le.numel() else 0)


class Paged:
    """A random paged cache with its sequences; slots that no sequence owns hold NaN."""

    def __init__(self, dtype, d, Hkv, page, lens, seed, order="token", spare=3, width=None):
        dev = "cuda"
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lens, self.page, self.d, self.Hkv = lens, page, d, Hkv
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        shape = (total, page, Hkv, d) if order == "token" else (total, Hkv, page, d)
        self.k = torch.full(shape, math.nan, dtype=dtype, device=dev)
        self.v = torch.full(shape, math.nan, dtype=dtype, device=dev)
        if order != "token":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        perm = torch.randperm(total, generator=g, device=dev).int()
        width = max(need + [1]) if width is None else width
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32, device=dev)   # never followed
        at = 0
        for s, c in enumerate(need):
            self.table[s, :c] = perm[at:at + c]
            at += c
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=dev)
        for s, n in enumerate(lens):
            self.put(s, torch.randn(n, Hkv, d, generator=g, device=dev).to(dtype), torch.randn(n, Hkv, d, generator=g, device=dev).to(dtype))

    def slots(self, s, keys):
        return self.table[s].long()[keys // self.page], keys % self.page

    def put(self, s, k, v):
        keys = torch.arange(k.shape[0], device="cuda")
        pg, sl = self.slots(s, keys)
        self.k[pg, sl], self.v[pg, sl] = k, v

    def get(self, s, n=None):
        keys = torch.arange(self.lens[s] if n is None else n, device="cuda")
        pg, sl = self.slots(s, keys)
        return self.k[pg, sl], self.v[pg, sl]


def limits(n, length, block, device="cuda"):
    p = torch.arange(length - n, length, device=device)
    if block == 0:
        return torch.full((n,), length, device=device)
    lim = (torch.div(p, block, rounding_mode="floor") + 1) * block
    return lim.clamp(0, length)


def cu_of(news, device="cuda"):
    return torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=device)
