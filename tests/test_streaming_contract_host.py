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


@pytest.mark.parametrize("ckw", [
    dict(v=FAKE + 16),                                                         # shifted by some channels
    dict(v=FAKE + 256),                                                        # by a head
    dict(v=FAKE + 1024),                                                       # by a token
    dict(v=FAKE + 16 * 1024),                                                  # by a page
    dict(k=FAKE + 16 * 1024, v=FAKE),
    dict(k_token=1024, k_page=16 * 1024, v_token=1024, v_page=16 * 1024, v=FAKE + 512),   # half a token's heads on
    dict(v=FAKE + 512, Hkv=4, k_head=256, k_token=1024, k_page=16 * 1024),
])
def test_append_refuses_caches_that_overlap(L, ckw):
    r = L.vdx_rope3d_append(ctypes.byref(_cache(**ckw)), ctypes.byref(_append()), None)
    assert r == B.VDX_ERR_ARG and "caches overlap" in L.vdx_last_error().decode(), L.vdx_last_error()


@pytest.mark.parametrize("ckw", [
    dict(v=FAKE + 1024, k_token=1024, k_page=16 * 1024, v_token=1024, v_page=16 * 1024),          # [pages, token, 2, H, d]
    dict(v=FAKE + 256, k_head=256, k_token=1024, k_page=16 * 1024, v_head=256, v_token=1024, v_page=16 * 1024),   # [.., H, 2, d]
    dict(v=FAKE + 16 * 1024, k_page=2 * 16 * 512, v_page=2 * 16 * 512),                           # [pages, 2, token, H, d]
    dict(v=FAKE + 20 * 16 * 1024),                                             # one right behind the other
])
def test_append_takes_caches_side_by_side(L, ckw):
    # refused only for what is checked after the caches: q and k of the call lie in the key cache
    r = L.vdx_rope3d_append(ctypes.byref(_cache(**ckw)), ctypes.byref(_append(k=FAKE + 16)), None)
    assert r == B.VDX_ERR_ARG and "the cache overlaps q, k, v or q_out" in L.vdx_last_error().decode(), L.vdx_last_error()


def test_paged_attention_checks_its_position_offsets(L):
    r = L.vdx_paged_attn_offset(ctypes.byref(_cache()), ctypes.byref(_paged()), FAKE + 9 * G + 2, None)
    assert r == B.VDX_ERR_ALIGN and "pos_offset" in L.vdx_last_error().decode(), L.vdx_last_error()


# ------------------------------------------------------------------------------------------ the build
@pytest.fixture
def small_build(tmp_path, monkeypatch):
    # one source, linked elsewhere: what build() does, in seconds
    monkeypatch.setattr(_build, "SOURCES", ["kv_capi.cu"])
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path / "out"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "EXT", str(tmp_path / "ext.so"))
    monkeypatch.setattr(_build, "EXT_STAMP", str(tmp_path / "ext.torch"))
    return tmp_path


def test_the_library_is_built_without_what_the_python_entry_needs(small_build, monkeypatch):
    base = small_build / "torch"                                   # a PyTorch without CUDA
    (base / "lib").mkdir(parents=True)
    (base / "__init__.py").write_text("")
    monkeypatch.setattr(_build.importlib.util, "find_spec",
                        lambda name: type("Spec", (), {"origin": str(base / "__init__.py")}))
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB) and not os.path.exists(_build.EXT)
    assert not _build._stale() and "no CUDA part" in _build._ext_lacks(str(base))
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
    assert not _build._stale() and "not installed" in _build._ext_lacks(None)


def test_a_python_without_headers_builds_the_library(small_build, monkeypatch):
    paths = dict(_build.sysconfig.get_paths(), include=str(small_build))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: paths)
    assert _build.build() == _build.LIB and not os.path.exists(_build.EXT) and not _build._stale()


def test_an_entry_that_does_not_compile_leaves_the_library(small_build, monkeypatch):
    def fails(torch):
        raise RuntimeError("does not compile")
    monkeypatch.setattr(_build, "_build_ext", fails)
    with pytest.raises(RuntimeError, match="does not compile"):
        _build.build()
    assert os.path.exists(_build.LIB)


# ------------------------------------------------------------------------- outputs over what the calls read beside q, k, v
@pytest.mark.parametrize("ckw,kw", [
    (dict(), dict(q_out=FAKE + 7 * G)),                                        # cu
    (dict(), dict(q_out=FAKE + 8 * G - 7 * 1024 + 16)),                        # kv_len, at q_out's end
    (dict(), dict(pos_offset=FAKE + 64)),
    (dict(page_table=FAKE + G + 1024), dict()),
    (dict(page_table=FAKE - 4 * (2 * 8 + 8) + 4), dict()),                     # the last page of the last sequence
    (dict(), dict(q_norm=FAKE + 6 * G + 512)),
    (dict(), dict(k_norm=FAKE - 240)),
])
def test_append_refuses_outputs_over_lengths_tables_and_weights(L, ckw, kw):
    r = L.vdx_rope3d_append(ctypes.byref(_cache(**ckw)), ctypes.byref(_append(**kw)), None)
    assert r == B.VDX_ERR_ARG and "overlaps cu, kv_len" in L.vdx_last_error().decode(), L.vdx_last_error()


def test_paged_attention_refuses_outputs_over_its_position_offsets(L):
    for out in (FAKE + 4 * G, FAKE + 5 * G):                       # out, lse
        r = L.vdx_paged_attn_offset(ctypes.byref(_cache()), ctypes.byref(_paged(causal_block=3)), out + 4, None)
        assert r == B.VDX_ERR_ARG and "overlaps cu, kv_len" in L.vdx_last_error().decode(), L.vdx_last_error()


@pytest.mark.parametrize("ckw,kw", [
    (dict(), dict(out=FAKE + 7 * G)), (dict(), dict(lse=FAKE + 8 * G)),
    (dict(page_table=FAKE + 5 * G + 7 * 4 * 4 - 4), dict()),
    (dict(page_table=FAKE + 4 * G - 4 * (2 * 8 + 8) + 4), dict()),
])
def test_paged_attention_refuses_outputs_over_lengths_and_tables(L, ckw, kw):
    r = L.vdx_paged_attn(ctypes.byref(_cache(**ckw)), ctypes.byref(_paged(**kw)), None)
    assert r == B.VDX_ERR_ARG and "overlaps cu, kv_len" in L.vdx_last_error().decode(), L.vdx_last_error()


def test_attention_refuses_scratch_and_outputs_over_lengths(L):
    c = _cache(page_size=128, max_pages=512, table_stride=512, num_pages=600, k_page=128 * 512, v_page=128 * 512)
    need = L.vdx_paged_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(_paged(rows=3, max_q=1)))
    assert need > 0
    for at in (FAKE + 7 * G, FAKE + 8 * G - need + 16, FAKE + 2 * G + 16):
        at -= at % 16
        a = _paged(rows=3, max_q=1, workspace=at, workspace_bytes=need)
        assert L.vdx_paged_attn(ctypes.byref(c), ctypes.byref(a), None) == B.VDX_ERR_ARG
        assert "overlaps cu, kv_len" in L.vdx_last_error().decode(), L.vdx_last_error()
    for kw in (dict(kv_len=FAKE + 3 * G + 64), dict(kv_len=FAKE + 4 * G)):
        assert L.vdx_cross_attn(ctypes.byref(_cross(**kw)), None) == B.VDX_ERR_ARG
        assert "overlaps cu, kv_len" in L.vdx_last_error().decode(), L.vdx_last_error()


def test_a_table_stride_past_its_bound_is_refused(L):
    c = _cache(table_stride=1 << 61)
    for r in (L.vdx_rope3d_append(ctypes.byref(c), ctypes.byref(_append()), None), L.vdx_paged_attn(ctypes.byref(c), ctypes.byref(_paged()), None)):
        assert r == B.VDX_ERR_ARG and "table_stride" in L.vdx_last_error().decode(), L.vdx_last_error()


def test_parameters_whose_products_are_not_finite_are_refused(L):
    r = L.vdx_rope3d_append(ctypes.byref(_cache()), ctypes.byref(_append(theta=5e-324)), None)
    assert r == B.VDX_ERR_ARG and "theta" in L.vdx_last_error().decode(), L.vdx_last_error()
    for r in (L.vdx_paged_attn(ctypes.byref(_cache()), ctypes.byref(_paged(scale=3e38)), None),
              L.vdx_cross_attn(ctypes.byref(_cross(scale=3e38)), None)):
        assert r == B.VDX_ERR_ARG and "scale" in L.vdx_last_error().decode(), L.vdx_last_error()


def test_more_sequences_and_heads_than_a_launch_has_blocks_are_refused(L):
    c = _cache(seqs=1 << 30, max_pages=1, table_stride=1)
    for r in (L.vdx_paged_attn(ctypes.byref(c), ctypes.byref(_paged()), None), L.vdx_cross_attn(ctypes.byref(_cross(B=1 << 29)), None)):
        assert r == B.VDX_ERR_ARG and "too many" in L.vdx_last_error().decode(), L.vdx_last_error()
