"""A NaN code of an 8-bit cache is NaN for every kernel that reads it, whatever the call's type."""
import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from kv8_ref import Paged8
from streaming_ref import DT, cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [3, 70], ids=["few-rows", "tiles"])
@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_a_nan_key_gathers_nan_from_rows_of_finite_lse(dtype, d, n, code):
    L, H, page = 600, 2, 32
    c = Paged8(d, H, page, [L], 301)
    g = torch.Generator(device="cuda").manual_seed(302)
    q = torch.randn(n, 2 * H, d, generator=g, device="cuda").to(DT[dtype])
    _, lse = vdx.paged_attn(q, c.cache(vdx), cu_of([n]), c.kv_len, causal_block=1)
    want = torch.zeros(1, H, L, device="cuda")
    vdx.paged_attn_weights(q, c.cache(vdx), cu_of([n]), c.kv_len, lse, want, causal_block=1)
    broken = [(0, 5, 0), (1, 131, d - 1), (1, 256, 17), (0, L - n, 3), (1, L - 1, d // 2 + 2)]      # head, key, channel
    k = c.k.view(torch.uint8)
    for h, key, ch in broken:
        page_of, slot = c.spots(0, key, 1)
        k[page_of, slot, h, ch] = code
    got = torch.zeros_like(want)
    vdx.paged_attn_weights(q, c.cache(vdx), cu_of([n]), c.kv_len, lse, got, causal_block=1)
    vdx.sync_check()
    assert bool(lse.isfinite().all()) and bool(want.isfinite().all())
    for h, key, _ in broken:
        assert bool(got[0, h, key].isnan()), (h, key, float(got[0, h, key]))
        got[0, h, key] = want[0, h, key]
    assert torch.equal(got, want)


def test_codes_of_both_kinds_are_their_values_in_bf16():
    # every code at every scale against its value: a single query channel of 1 picks it out, lse takes the score back to 0
    d, L, H, page, n = 64, 256, 1, 16, 40
    c = Paged8(d, H, page, [L], 303)
    q = torch.zeros(n, 1, d, device="cuda", dtype=torch.bfloat16)
    q[:, 0, 7] = 1
    bits, sc = c.k.view(torch.uint8), c.k_scale.view(torch.uint8)
    page_of, slot = c.spots(0, 0, L)
    codes = torch.arange(L, dtype=torch.uint8, device="cuda")
    bits[page_of, slot, 0] = 0
    bits[page_of, slot, 0, 7] = codes
    for e in (-15, -8, -6):                                # larger scales: 2^x of the larger codes is past fp32
        sc[page_of, slot // 16, 0] = e + 127
        value = codes.view(torch.float8_e4m3fn).float().double() * 2.0 ** e
        w = torch.zeros(1, 1, L, device="cuda")
        vdx.paged_attn_weights(q, c.cache(vdx), cu_of([n]), c.kv_len, torch.zeros(1, n, device="cuda"), w, scale=1.0)
        vdx.sync_check()
        want = n * torch.exp(value)
        # the scale's two roundings to log2 units and the product's (2^-22 of the exponent), the exponential, a sum of n
        bound = want * (2.0 ** -22 * value.abs() + 2.0 ** -21 + n * 2.0 ** -23)
        nan = value.isnan()
        assert int(nan.sum()) == 2 and torch.equal(w[0, 0].isnan(), nan)
        assert bool(((w[0, 0].double() - want).abs() <= bound)[~nan].all())
