"""The 8-bit cache, gathered weights and eviction without a GPU: every refusal happens before any CUDA call (the
addresses below are never dereferenced), and the binding's structures match include/vdx.h."""
import ctypes
import os
import re
import subprocess

import pytest

import video_diffusion_transformer_rope_gb300 as vdx
from video_diffusion_transformer_rope_gb300 import _binding as B
from video_diffusion_transformer_rope_gb300 import _build
from test_streaming_host import CACHE_REFUSALS, FAKE, G, L, ROOT, _append, _cache, _paged  # noqa: F401

S = FAKE + 20 * G


def _scales(**kw):
    d = dict(k=S, v=S + G, k_page=4, k_block=4, k_head=1, v_page=4, v_block=4, v_head=1)
    d.update(kw)
    return B.Kv8Scales(**d)


def _weights(**kw):
    d = dict(q=FAKE + 3 * G, lse=FAKE + 5 * G, w=FAKE + 10 * G, q_row=512, q_head=128, w_seq=4 * 128, w_head=128, width=128, rows=7, Hq=4,
             cu=FAKE + 7 * G, kv_len=FAKE + 8 * G, pos_offset=0, max_q=0, max_kv=0, causal_block=0, scale=0.0, decay=1.0)
    d.update(kw)
    return B.PagedWeightsArgs(**d)


def _evict(**kw):
    d = dict(w=FAKE + 10 * G, w_out=FAKE + 11 * G, w_seq=4 * 128, w_head=128, w_out_seq=4 * 50, w_out_head=50, width=128,
             kv_len=FAKE + 8 * G, pos_offset=0, kv_len_out=FAKE + 12 * G, pos_offset_out=FAKE + 13 * G, index=FAKE + 14 * G, keep=50,
             recent=3, max_kv=0)
    d.update(kw)
    return B.PagedEvictArgs(**d)


def _to(**kw):
    return _cache(**dict(dict(k=FAKE + 30 * G, v=FAKE + 31 * G, page_table=FAKE + 32 * G), **kw))


def _to_scales(**kw):
    return _scales(**dict(dict(k=S + 2 * G, v=S + 3 * G), **kw))


def _refused(L, r, status, msg):
    assert r == status and msg in L.vdx_last_error().decode(), (r, L.vdx_last_error())


ref = ctypes.byref


@pytest.mark.parametrize("kw,status,msg", CACHE_REFUSALS)
def test_cache_refusals_hold_for_every_call(L, kw, status, msg):
    if kw == dict(k_token=516):
        kw, msg = dict(k_token=520), "multiple of 16"
    c, s = _cache(**kw), _scales()
    _refused(L, L.vdx_rope3d_append8(ref(c), ref(s), ref(_append()), None), status, msg)
    _refused(L, L.vdx_paged_attn8(ref(c), ref(s), ref(_paged()), None, None), status, msg)
    assert L.vdx_paged_attn8_workspace_bytes(ref(c), ref(s), ref(_paged())) == 0 and L.vdx_last_error()
    _refused(L, L.vdx_paged_attn_weights(ref(c), ref(s), ref(_weights()), None), status, msg)
    if msg != "multiple":                               # eviction has no query heads
        _refused(L, L.vdx_paged_evict(ref(c), ref(s), ref(_to()), ref(_to_scales()), ref(_evict()), None), status, msg)
        _refused(L, L.vdx_paged_evict(ref(_to()), ref(_to_scales()), ref(c), ref(s), ref(_evict()), None), status, msg)


SCALE_REFUSALS = [
    (dict(k=0), "non-NULL"), (dict(v=0), "non-NULL"), (dict(k_page=0), "stride"), (dict(v_head=-1), "stride"),
    (dict(v_page=1 << 39), "stride"),
]


@pytest.mark.parametrize("kw,msg", SCALE_REFUSALS)
def test_scale_refusals(L, kw, msg):
    s = _scales(**kw)
    _refused(L, L.vdx_rope3d_append8(ref(_cache()), ref(s), ref(_append()), None), B.VDX_ERR_ARG, msg)
    _refused(L, L.vdx_paged_attn8(ref(_cache()), ref(s), ref(_paged()), None, None), B.VDX_ERR_ARG, msg)
    _refused(L, L.vdx_paged_attn_weights(ref(_cache()), ref(s), ref(_weights()), None), B.VDX_ERR_ARG, msg)
    _refused(L, L.vdx_paged_evict(ref(_cache()), ref(s), ref(_to()), ref(_to_scales()), ref(_evict()), None), B.VDX_ERR_ARG, msg)


def test_calls_of_8_bits_need_scales(L):
    _refused(L, L.vdx_rope3d_append8(ref(_cache()), None, ref(_append()), None), B.VDX_ERR_ARG, "scales must be")
    _refused(L, L.vdx_paged_attn8(ref(_cache()), None, ref(_paged()), None, None), B.VDX_ERR_ARG, "scales must be")
    assert L.vdx_paged_attn8_workspace_bytes(ref(_cache()), None, ref(_paged())) == 0 and b"scales" in L.vdx_last_error()


@pytest.mark.parametrize("kw,msg", [
    (dict(k_head=1, k_block=2, k_page=2), "overlap one another"), (dict(v=S + 3), "key and value scales overlap"),
    (dict(k=FAKE + 64), "scales overlap the cache"), (dict(v=FAKE + 4 * G + 8), "overlap q, k, v"),
    (dict(v=FAKE + 6 * G + 8), "overlap q, k, v"), (dict(k=FAKE + 7 * G + 4), "overlap cu"), (dict(k=FAKE + 8 * G - 70), "overlap cu"),
    (dict(v=FAKE + 2 * G), "overlap cu"),
])
def test_append_refuses_scales_over_other_memory(L, kw, msg):
    _refused(L, L.vdx_rope3d_append8(ref(_cache()), ref(_scales(**kw)), ref(_append()), None), B.VDX_ERR_ARG, msg)


def test_scales_side_by_side_are_taken(L):
    # [pages, blocks, 2, heads]; refused only for what is checked afterwards
    s = _scales(v=S + 4, k_page=8, k_block=8, v_page=8, v_block=8)
    _refused(L, L.vdx_rope3d_append8(ref(_cache()), ref(s), ref(_append(q_norm=FAKE + 6 * G + 512)), None), B.VDX_ERR_ARG, "overlaps cu")
    s = _scales(v=FAKE + 7 * G - 4, k_page=8, k_block=8, v_page=8, v_block=8, k=FAKE + 7 * G - 8)
    _refused(L, L.vdx_rope3d_append8(ref(_cache()), ref(s), ref(_append()), None), B.VDX_ERR_ARG, "scales overlap cu")


@pytest.mark.parametrize("kw", [dict(out=S + 16), dict(lse=S + G + 16), dict(out=S - 7 * 4 * 128 * 2 + 16)])
def test_attention_refuses_outputs_over_scales(L, kw):
    _refused(L, L.vdx_paged_attn8(ref(_cache()), ref(_scales()), ref(_paged(**kw)), None, None), B.VDX_ERR_ARG, "overlaps the scales")


@pytest.mark.parametrize("kw,status,msg", [
    (dict(rows=-1), B.VDX_ERR_ARG, "rows"), (dict(max_q=-1), B.VDX_ERR_ARG, "max_q"), (dict(causal_block=-1), B.VDX_ERR_ARG, "causal_block"),
    (dict(width=-1), B.VDX_ERR_ARG, "width"), (dict(decay=float("inf")), B.VDX_ERR_ARG, "decay"), (dict(scale=float("nan")), B.VDX_ERR_ARG, "scale"),
    (dict(scale=3e38), B.VDX_ERR_ARG, "too large"), (dict(lse=0), B.VDX_ERR_ARG, "lse"), (dict(lse=FAKE + 5 * G + 2), B.VDX_ERR_ALIGN, "lse"),
    (dict(w=0), B.VDX_ERR_ARG, "weights"), (dict(w=FAKE + 10 * G + 1), B.VDX_ERR_ALIGN, "weights"), (dict(w_head=127), B.VDX_ERR_ARG, "stride"),
    (dict(w_seq=500), B.VDX_ERR_ARG, "overlap one another"), (dict(cu=0), B.VDX_ERR_ARG, "cu"), (dict(kv_len=FAKE + 8 * G + 2), B.VDX_ERR_ALIGN, "kv_len"),
    (dict(pos_offset=FAKE + 2), B.VDX_ERR_ALIGN, "pos_offset"), (dict(q=0), B.VDX_ERR_ARG, "q must"), (dict(q_row=100), B.VDX_ERR_ARG, "stride"),
    (dict(Hq=6), B.VDX_ERR_ARG, "multiple"), (dict(w=FAKE + 3 * G + 64), B.VDX_ERR_ARG, "overlap q or the cache"),
    (dict(w=FAKE + 512), B.VDX_ERR_ARG, "overlap q or the cache"), (dict(w=S), B.VDX_ERR_ARG, "overlap q or the cache"),
    (dict(w=FAKE + 5 * G), B.VDX_ERR_ARG, "overlap cu"), (dict(w=FAKE + 7 * G), B.VDX_ERR_ARG, "overlap cu"),
    (dict(w=FAKE + 8 * G - 1000), B.VDX_ERR_ARG, "overlap cu"), (dict(w=FAKE + 2 * G), B.VDX_ERR_ARG, "overlap cu"),
    (dict(causal_block=2, pos_offset=FAKE + 10 * G + 4), B.VDX_ERR_ARG, "overlap cu"),
])
def test_weights_refusals(L, kw, status, msg):
    _refused(L, L.vdx_paged_attn_weights(ref(_cache()), ref(_scales()), ref(_weights(**kw)), None), status, msg)


def test_calls_with_nothing_to_do_are_taken(L):
    for s in (None, ref(_scales())):
        assert L.vdx_paged_attn_weights(ref(_cache()), s, ref(_weights(rows=0, q=0, lse=0, w=0)), None) == B.VDX_OK
        assert L.vdx_paged_attn_weights(ref(_cache(seqs=0)), s, ref(_weights()), None) == B.VDX_OK
    assert L.vdx_paged_evict(ref(_cache(seqs=0)), None, ref(_to(seqs=0)), None, ref(_evict()), None) == B.VDX_OK
    assert L.vdx_rope3d_append8(ref(_cache()), ref(_scales()), ref(_append(rows=0)), None) == B.VDX_OK
    assert L.vdx_paged_attn8(ref(_cache()), ref(_scales()), ref(_paged(rows=0)), None, None) == B.VDX_OK


@pytest.mark.parametrize("kw,status,msg", [
    (dict(keep=0), B.VDX_ERR_ARG, "keep"), (dict(recent=-1), B.VDX_ERR_ARG, "recent"), (dict(recent=51), B.VDX_ERR_ARG, "recent"),
    (dict(width=-1), B.VDX_ERR_ARG, "width"), (dict(max_kv=-1), B.VDX_ERR_ARG, "max_kv"), (dict(keep=1 << 30), B.VDX_ERR_ARG, "too large"),
    (dict(w=0), B.VDX_ERR_ARG, "w must"), (dict(w_out=0), B.VDX_ERR_ARG, "w_out must"), (dict(w_out=FAKE + 11 * G + 2), B.VDX_ERR_ALIGN, "w_out"),
    (dict(w_head=100), B.VDX_ERR_ARG, "stride"), (dict(w_out_seq=150), B.VDX_ERR_ARG, "overlap one another"), (dict(w_out_head=49), B.VDX_ERR_ARG, "stride"),
    (dict(kv_len=0), B.VDX_ERR_ARG, "kv_len"), (dict(kv_len_out=0), B.VDX_ERR_ARG, "kv_len_out"), (dict(index=0), B.VDX_ERR_ARG, "index"),
    (dict(pos_offset_out=FAKE + 13 * G + 1), B.VDX_ERR_ALIGN, "pos_offset_out"),
    (dict(w_out=FAKE + 10 * G), B.VDX_ERR_ARG, "other strides"), (dict(w_out=FAKE + 10 * G, w_out_seq=512, w_out_head=128, keep=129, recent=0), B.VDX_ERR_ARG, "smaller than keep"),
    (dict(w_out=FAKE + 10 * G + 4, w_out_seq=512, w_out_head=128), B.VDX_ERR_ARG, "w_out overlaps w"),
    (dict(kv_len_out=FAKE + 8 * G), B.VDX_ERR_ARG, "overlaps kv_len"), (dict(index=FAKE + 32 * G), B.VDX_ERR_ARG, "overlaps kv_len"),
    (dict(index=FAKE + 12 * G), B.VDX_ERR_ARG, "overlap one another"), (dict(index=FAKE + 10 * G), B.VDX_ERR_ARG, "overlaps w"),
    (dict(kv_len_out=FAKE + 11 * G), B.VDX_ERR_ARG, "overlaps w"), (dict(index=FAKE + 30 * G), B.VDX_ERR_ARG, "overlaps a cache"),
    (dict(w_out=FAKE + 8 * G), B.VDX_ERR_ARG, "w_out overlaps kv_len"), (dict(w_out=FAKE + 64), B.VDX_ERR_ARG, "w_out overlaps a cache"),
    (dict(w=FAKE + 31 * G), B.VDX_ERR_ARG, "w overlaps the cache"), (dict(w_out=S + 4), B.VDX_ERR_ARG, "scales overlap w"),
    (dict(w=S + 2 * G), B.VDX_ERR_ARG, "scales overlap w"), (dict(kv_len_out=S + 3 * G), B.VDX_ERR_ARG, "scales overlap kv_len_out"),
    (dict(kv_len=S + 2 * G), B.VDX_ERR_ARG, "scales overlap kv_len,"),
])
def test_evict_refusals(L, kw, status, msg):
    _refused(L, L.vdx_paged_evict(ref(_cache()), ref(_scales()), ref(_to()), ref(_to_scales()), ref(_evict(**kw)), None), status, msg)


def test_evict_says_how_many_keys_it_takes(L):
    big = dict(page_size=1 << 14, max_pages=25, table_stride=25, num_pages=30, k_page=1 << 23, v_page=1 << 23)
    c, to = _cache(**big), _to(**dict(big, k=FAKE + 30 * G, v=FAKE + 31 * G))
    a = dict(w_head=1 << 19, w_seq=1 << 21, width=1 << 19)
    _refused(L, L.vdx_paged_evict(ref(c), None, ref(to), None, ref(_evict(**a)), None), B.VDX_ERR_UNSUPPORTED, "393216 keys")


@pytest.mark.parametrize("tkw,msg", [
    (dict(Hkv=3), "one kind"), (dict(d=64), "one kind"), (dict(dtype=1), "one kind"), (dict(seqs=2), "one kind"),
    (dict(k=FAKE, v=FAKE + G, page_table=FAKE + 2 * G), "same page table"), (dict(k=FAKE, v=FAKE + G, num_pages=19), "same strides"),
    (dict(k=FAKE, v=FAKE + G, k_token=1024, k_page=16 * 1024), "same strides"), (dict(k=FAKE), "overlap without"),
    (dict(v=FAKE + 512), "overlap without"), (dict(k=FAKE + G, v=FAKE), "overlap without"), (dict(v=FAKE + 30 * G), "same memory"),
])
def test_evict_refuses_caches_that_do_not_go_together(L, tkw, msg):
    _refused(L, L.vdx_paged_evict(ref(_cache()), None, ref(_to(**tkw)), None, ref(_evict()), None), B.VDX_ERR_ARG, msg)


@pytest.mark.parametrize("skw,msg", [
    (dict(k=S), "scales of the two caches"), (dict(k=S + G), "scales of the two caches"), (dict(v=S + 2 * G), "value scales overlap"),
    (dict(k=FAKE + 512), "scales overlap a cache"), (dict(v=FAKE + 30 * G), "scales overlap the cache"),
])
def test_evict_refuses_scales_over_other_memory(L, skw, msg):
    _refused(L, L.vdx_paged_evict(ref(_cache()), ref(_scales()), ref(_to()), ref(_to_scales(**skw)), ref(_evict()), None), B.VDX_ERR_ARG, msg)
    _refused(L, L.vdx_paged_evict(ref(_cache()), ref(_scales()), ref(_to()), None, ref(_evict()), None), B.VDX_ERR_ARG, "one kind")


def test_structures_match_the_header(tmp_path):
    pairs = {"vdx_kv8_scales": B.Kv8Scales, "vdx_paged_weights_args": B.PagedWeightsArgs, "vdx_paged_evict_args": B.PagedEvictArgs}
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "vdx.h"', 'int main(void) {']
    for name, st in pairs.items():
        src.append(f'printf("{name} %zu\\n", sizeof({name}));')
        src += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in st._fields_]
    src.append('printf("block %d\\n", VDX_KV8_BLOCK); return 0; }')
    (tmp_path / "o.c").write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["block"]) == vdx.KV8_BLOCK
    for name, st in pairs.items():
        assert int(got[name]) == ctypes.sizeof(st)
        for f in st._fields_:
            assert int(got[f"{name}.{f[0]}"]) == getattr(st, f[0]).offset


@pytest.mark.parametrize("name", ["kv8.cuh", "kv_mma.cuh", "rows_join.cuh", "attn_rows8.cu", "kv_weigh.cu", "weigh_tiles_sm103.cu", "sm103_wait.cuh", "kv_evict.cu"])
def test_kernels_that_start_early_read_through_the_coherent_path(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__|ld_nc", text)


def test_python_refuses_host_tensors():
    import torch
    t = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16)
    cache = vdx.PagedKV(t, t, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(vdx.VdxError):
        vdx.paged_attn_weights(t[0], cache, None, None, None, None)
    with pytest.raises(vdx.VdxError):
        vdx.paged_evict(cache, None, None, 1, cache)
