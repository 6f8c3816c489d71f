"""What sync_check says of calls over paged caches: the message is of the call that was made."""
import pytest
import torch

import video_diffusion_transformer_rope_gb300 as vdx
from streaming_ref import Paged, cu_of

pytestmark = pytest.mark.gpu


def _cache(lens, seed):
    c = Paged(torch.bfloat16, 64, 2, 16, lens, seed, order="head")
    return c, vdx.PagedKV(c.k, c.v, c.table)


def test_a_page_table_too_short_to_evict_into_is_named():
    c, cache = _cache([40, 30], 401)
    into, _ = _cache([20, 20], 402)
    short = vdx.PagedKV(into.k, into.v, into.table[:, :1].contiguous())
    vdx.paged_evict(cache, torch.rand(2, 2, 48, device="cuda"), c.kv_len, 20, short)
    with pytest.raises(vdx.VdxError, match="eviction") as e:
        vdx.sync_check()
    assert "append" not in str(e.value)
    vdx.sync_check()


@pytest.mark.parametrize("n", [2, 33, 300])
def test_lengths_past_weights_of_no_width_are_reported_whatever_the_rows(n):
    c, cache = _cache([400, 310], 403)
    q = torch.randn(2 * n, 4, 64, device="cuda").to(torch.bfloat16)
    lse = torch.zeros(4, 2 * n, device="cuda")
    none = torch.zeros(2, 2, 0, device="cuda")
    vdx.paged_attn_weights(q, cache, cu_of([n, n]), c.kv_len, lse, none)
    with pytest.raises(vdx.VdxError, match="kv_len"):
        vdx.sync_check()
    vdx.paged_attn_weights(q, cache, cu_of([n, n]), torch.zeros_like(c.kv_len), lse, none)
    vdx.sync_check()
