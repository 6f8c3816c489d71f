"""Refusals of gathered weights that test_kv8_host.py does not make; nothing here reaches CUDA."""
import ctypes

import pytest

from video_diffusion_transformer_rope_gb300 import _binding as B
from test_kv8_host import _refused, _weights
from test_streaming_host import L, _cache  # noqa: F401

ref = ctypes.byref


@pytest.mark.parametrize("rows,max_q,Hq,taken", [
    ((1 << 26) + 1, 0, 4, False), ((1 << 26) + 1, 1 << 26, 4, True), (1 << 26, 0, 4, True), ((1 << 24) + 1, 0, 16, False), (1 << 24, 0, 16, True),
    (1 << 28, 1 << 19, 512, True), (1 << 28, (1 << 19) + 1, 512, False),
])
def test_rows_that_the_tile_kernel_could_not_finish_in_its_waits_are_refused(L, rows, max_q, Hq, taken):
    a = _weights(rows=rows, max_q=max_q, Hq=Hq, q_row=128 * Hq, cu=0)                      # taken: refused for what comes after
    _refused(L, L.vdx_paged_attn_weights(ref(_cache()), None, ref(a), None), B.VDX_ERR_ARG if taken else B.VDX_ERR_UNSUPPORTED,
             "cu must" if taken else "rows per kv head")
