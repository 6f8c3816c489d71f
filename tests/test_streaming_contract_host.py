"""Promises of the paged-cache and cross-attention calls that can be checked without a GPU: refusals before any
CUDA call (the addresses are never dereferenced), and rules that their kernels' sources keep."""
import ctypes
import os
import re

import pytest

from video_diffusion_transformer_rope_gb300 import _binding as B
from video_diffusion_transformer_rope_gb300 import _build
from test_streaming_host import FAKE, G, L, _append, _cache, _cross, _paged  # noqa: F401

KERNELS = ["kv_common.cuh", "kv_append.cu", "attn_rows.cu", "attn_tiles_sm103.cu"]


def _source(name):
    text = open(os.path.join(_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", KERNELS)
def test_kernels_that_start_early_read_through_the_coherent_path(name):
    # the work before a call may still be writing its inputs when the kernel starts: a load of the read-only path
    # (also one that the compiler may choose, given const __restrict__) need not see them after the wait
    text = _source(name)
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__|ld_nc", text)


def test_arrivals_released_to_the_cluster_are_waited_for_at_cluster_scope():
    # a barrier on which the other CTA arrives with a cluster-scope release (it announces plain stores or reads)
    # has a wait whose acquire has that scope too; one of CTA scope does not pair with it
    text = _source("attn_tiles_sm103.cu")
    bars = set(re.findall(r"mbar_arrive_remote_cluster\((?:mapa_shared\(sCtl \+|remote \+) (kBar\w+)", text))
    assert bars == {"kBarVFull", "kBarClaimReady"}
    for bar in bars:
        assert re.search(r"warp_wait<true>\(sCtl \+ %s\b" % bar, text), bar
