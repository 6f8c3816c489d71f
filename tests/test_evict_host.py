"""Refusals of eviction that test_kv8_host.py does not make; nothing here reaches CUDA."""
import ctypes

import pytest

from video_diffusion_transformer_rope_gb300 import _binding as B
from test_kv8_host import _evict, _refused, _to
from test_streaming_host import FAKE, G, L, _cache  # noqa: F401

ref = ctypes.byref


# [3, 4, 128] weights with heads 128 apart whose sequences begin inside the one before: as read-only weights they are taken, but
# written in place the 40 of one head would lie over another's that are still to be read.
@pytest.mark.parametrize("seq", [3 * 128 + 40, 511])
def test_weights_in_place_may_not_overlap_one_another(L, seq):
    same = _evict(w_out=FAKE + 10 * G, w_seq=seq, w_out_seq=seq, w_head=128, w_out_head=128, keep=40, recent=3)
    _refused(L, L.vdx_paged_evict(ref(_cache()), None, ref(_to()), None, ref(same), None), B.VDX_ERR_ARG, "rows of w overlap one another")
    apart = _evict(w_seq=seq, keep=40, w_out_seq=160, w_out_head=40, kv_len_out=0)         # refused for what comes after
    _refused(L, L.vdx_paged_evict(ref(_cache()), None, ref(_to()), None, ref(apart), None), B.VDX_ERR_ARG, "kv_len_out")
    whole = _evict(w_out=FAKE + 10 * G, w_out_seq=512, w_out_head=128, keep=40, kv_len_out=0)
    _refused(L, L.vdx_paged_evict(ref(_cache()), None, ref(_to()), None, ref(whole), None), B.VDX_ERR_ARG, "kv_len_out")
