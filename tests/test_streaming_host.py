"""Paged-cache and cross-attention calls: every refusal happens before any CUDA call (no GPU here;
the addresses below are never dereferenced), and the binding's structures match include/vdx.h."""
import ctypes
import os
import re
import subprocess

import pytest

import video_diffusion_transformer_rope_gb300 as vdx
from video_diffusion_transformer_rope_gb300 import _binding as B
from video_diffusion_transformer_rope_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 32
FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return vdx.lib()


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE + G, k_page=16 * 512, k_token=512, k_head=128, v_page=16 * 512, v_token=512, v_head=128,
             page_table=FAKE + 2 * G, table_stride=8, num_pages=20, page_size=16, max_pages=8, Hkv=4, d=128, dtype=0, seqs=3)
    d.update(kw)
    return B.PagedKvStruct(**d)


def _append(**kw):
    d = dict(q=FAKE + 3 * G, k=FAKE + 4 * G, v=FAKE + 5 * G, q_out=FAKE + 6 * G, q_row=512, q_head=128, k_row=512, k_head=128,
             v_row=512, v_head=128, q_out_row=512, q_out_head=128, rows=7, Hq=4, cu=FAKE + 7 * G, kv_len=FAKE + 8 * G,
             pos_offset=0, T=4, Hgrid=3, Wgrid=5, sec_t=0, sec_h=0, sec_w=0, theta=10000.0, q_norm=0, k_norm=0, eps=1e-6)
    d.update(kw)
    return B.AppendArgs(**d)


def _paged(**kw):
    d = dict(q=FAKE + 3 * G, out=FAKE + 4 * G, lse=FAKE + 5 * G, q_row=512, q_head=128, rows=7, Hq=4, cu=FAKE + 7 * G,
             kv_len=FAKE + 8 * G, max_q=0, max_kv=0, causal_block=0, scale=0.0, workspace=0, workspace_bytes=0)
    d.update(kw)
    return B.PagedAttnArgs(**d)


def _cross(**kw):
    d = dict(q=FAKE, k=FAKE + G, v=FAKE + 2 * G, out=FAKE + 3 * G, lse=FAKE + 4 * G, q_batch=5 * 512, q_row=512, q_head=128,
             k_batch=9 * 512, k_token=512, k_head=128, v_batch=9 * 512, v_token=512, v_head=128, B=2, N=5, M=9, Hq=4, Hkv=4,
             d=128, dtype=0, kv_len=0, scale=0.0, workspace=0, workspace_bytes=0)
    d.update(kw)
    return B.CrossAttnArgs(**d)


CACHE_REFUSALS = [
    (dict(dtype=2), B.VDX_ERR_ARG, "dtype"),
    (dict(d=96), B.VDX_ERR_UNSUPPORTED, "head_dim"),
    (dict(Hkv=0), B.VDX_ERR_ARG, "head counts"),
    (dict(Hkv=3), B.VDX_ERR_ARG, "multiple"),
    (dict(page_size=24), B.VDX_ERR_UNSUPPORTED, "page_size"),
    (dict(page_size=0), B.VDX_ERR_UNSUPPORTED, "page_size"),
    (dict(page_size=127), B.VDX_ERR_UNSUPPORTED, "page_size"),
    (dict(num_pages=0), B.VDX_ERR_ARG, "num_pages"),
    (dict(max_pages=0), B.VDX_ERR_ARG, "max_pages"),
    (dict(max_pages=1 << 27, table_stride=1 << 27), B.VDX_ERR_ARG, "too large"),
    (dict(seqs=-1), B.VDX_ERR_ARG, "seqs"),
    (dict(table_stride=7), B.VDX_ERR_ARG, "table_stride"),
    (dict(page_table=0), B.VDX_ERR_ARG, "page_table"),
    (dict(page_table=FAKE + 2 * G + 2), B.VDX_ERR_ALIGN, "page_table"),
    (dict(k=0), B.VDX_ERR_ARG, "key cache"),
    (dict(v=FAKE + G + 8), B.VDX_ERR_ALIGN, "value cache"),
    (dict(k_token=516), B.VDX_ERR_ARG, "multiple of 8"),
    (dict(k_head=0), B.VDX_ERR_ARG, "smaller"),
    (dict(v_page=0), B.VDX_ERR_ARG, "smaller"),
    (dict(k_page=-8), B.VDX_ERR_ARG, "stride"),
    (dict(v_head=1 << 39), B.VDX_ERR_ARG, "stride"),
]


@pytest.mark.parametrize("kw,status,msg", CACHE_REFUSALS)
def test_cache_refusals(L, kw, status, msg):
    c, a, p = _cache(**kw), _append(), _paged()
    for r in (L.vdx_rope3d_append(ctypes.byref(c), ctypes.byref(a), None), L.vdx_paged_attn(ctypes.byref(c), ctypes.byref(p), None)):
        assert r == status and msg in L.vdx_last_error().decode(), L.vdx_last_error()
    assert L.vdx_paged_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw,status,msg", [
    (dict(rows=-1), B.VDX_ERR_ARG, "rows"),
    (dict(q_out=0), B.VDX_ERR_ARG, "go together"),
    (dict(q=0), B.VDX_ERR_ARG, "go together"),
    (dict(q=0, q_out=0, q_norm=FAKE + 9 * G), B.VDX_ERR_ARG, "q_norm"),
    (dict(k=0), B.VDX_ERR_ARG, "k must be"),
    (dict(v=0), B.VDX_ERR_ARG, "v must be"),
    (dict(cu=0), B.VDX_ERR_ARG, "cu"),
    (dict(kv_len=0), B.VDX_ERR_ARG, "kv_len"),
    (dict(kv_len=FAKE + 8 * G + 1), B.VDX_ERR_ALIGN, "kv_len"),
    (dict(pos_offset=FAKE + 9 * G + 2), B.VDX_ERR_ALIGN, "pos_offset"),
    (dict(q=FAKE + 3 * G + 4), B.VDX_ERR_ALIGN, "q is not"),
    (dict(k_norm=FAKE + 9 * G + 8), B.VDX_ERR_ALIGN, "k_norm"),
    (dict(T=0), B.VDX_ERR_ARG, ">= 1"),
    (dict(Hgrid=1 << 20, Wgrid=1 << 20), B.VDX_ERR_ARG, "too large"),
    (dict(sec_t=43, sec_h=43, sec_w=42), B.VDX_ERR_ARG, "sections"),
    (dict(sec_t=40, sec_h=40, sec_w=40), B.VDX_ERR_ARG, "sections"),
    (dict(theta=0.0), B.VDX_ERR_ARG, "theta"),
    (dict(eps=-1.0), B.VDX_ERR_ARG, "eps"),
    (dict(eps=float("nan")), B.VDX_ERR_ARG, "eps"),
    (dict(Hq=6), B.VDX_ERR_ARG, "multiple"),
    (dict(q_out=FAKE + 3 * G + 256), B.VDX_ERR_ARG, "overlaps"),
    (dict(q_out=FAKE + 4 * G), B.VDX_ERR_ARG, "overlaps"),
    (dict(v=FAKE + G), B.VDX_ERR_ARG, "cache overlaps"),
    (dict(k_row=100), B.VDX_ERR_ARG, "stride"),
])
def test_append_refusals(L, kw, status, msg):
    r = L.vdx_rope3d_append(ctypes.byref(_cache()), ctypes.byref(_append(**kw)), None)
    assert r == status and msg in L.vdx_last_error().decode(), L.vdx_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(rows=-1), B.VDX_ERR_ARG, "rows"),
    (dict(max_q=-1), B.VDX_ERR_ARG, "max_q"),
    (dict(max_kv=-1), B.VDX_ERR_ARG, "max_kv"),
    (dict(causal_block=-1), B.VDX_ERR_ARG, "causal_block"),
    (dict(scale=float("inf")), B.VDX_ERR_ARG, "scale"),
    (dict(q=0), B.VDX_ERR_ARG, "q must be"),
    (dict(out=0), B.VDX_ERR_ARG, "out must be"),
    (dict(out=FAKE + 4 * G + 8), B.VDX_ERR_ALIGN, "out"),
    (dict(lse=FAKE + 5 * G + 2), B.VDX_ERR_ALIGN, "lse"),
    (dict(cu=0), B.VDX_ERR_ARG, "cu"),
    (dict(out=FAKE + 3 * G + 64), B.VDX_ERR_ARG, "out overlaps"),
    (dict(out=FAKE + 64), B.VDX_ERR_ARG, "out overlaps"),
    (dict(lse=FAKE + 4 * G + 64), B.VDX_ERR_ARG, "lse overlaps out"),
    (dict(lse=FAKE + G + 64), B.VDX_ERR_ARG, "lse overlaps q, k or v"),
    (dict(Hq=516), B.VDX_ERR_UNSUPPORTED, "128 query heads"),
    (dict(q_row=4), B.VDX_ERR_ARG, "stride"),
])
def test_paged_refusals(L, kw, status, msg):
    r = L.vdx_paged_attn(ctypes.byref(_cache()), ctypes.byref(_paged(**kw)), None)
    assert r == status and msg in L.vdx_last_error().decode(), L.vdx_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(B=-1), B.VDX_ERR_ARG, ">= 0"),
    (dict(M=-1), B.VDX_ERR_ARG, ">= 0"),
    (dict(M=1 << 30), B.VDX_ERR_ARG, "too large"),
    (dict(d=80), B.VDX_ERR_UNSUPPORTED, "head_dim"),
    (dict(dtype=-1), B.VDX_ERR_ARG, "dtype"),
    (dict(Hq=5, Hkv=2), B.VDX_ERR_ARG, "multiple"),
    (dict(q=0), B.VDX_ERR_ARG, "q must be"),
    (dict(v=0), B.VDX_ERR_ARG, "v must be"),
    (dict(k=FAKE + G + 4), B.VDX_ERR_ALIGN, "k is not"),
    (dict(k_token=0), B.VDX_ERR_ARG, "smaller"),
    (dict(q_row=0), B.VDX_ERR_ARG, "smaller"),
    (dict(kv_len=FAKE + 9 * G + 1), B.VDX_ERR_ALIGN, "kv_len"),
    (dict(out=FAKE), B.VDX_ERR_ARG, "out overlaps"),
    (dict(scale=float("nan")), B.VDX_ERR_ARG, "scale"),
])
def test_cross_refusals(L, kw, status, msg):
    r = L.vdx_cross_attn(ctypes.byref(_cross(**kw)), None)
    assert r == status and msg in L.vdx_last_error().decode(), L.vdx_last_error()


@pytest.mark.parametrize("ckw,kw,msg", [
    # rows or slots that lie over one another: two rows of the call would write one place
    (dict(), dict(q_out_row=384), "q_out"),
    (dict(), dict(q_out_row=128, q_out_head=128 * 6), "q_out"),
    (dict(k_token=384), dict(), "key cache"),
    (dict(v_page=15 * 512), dict(), "value cache"),
    (dict(v=FAKE), dict(), "same memory"),
    # q in place, and k or v in the rows that it turns
    (dict(), dict(q_out=FAKE + 3 * G, k=FAKE + 3 * G), "q_out overlaps"),
    (dict(), dict(q_out=FAKE + 3 * G, v=FAKE + 3 * G + 256), "q_out overlaps"),
    (dict(), dict(q_out=FAKE + 3 * G, q_row=1536, q_out_row=1536, k_row=1536, k=FAKE + 3 * G + 1024 - 256), "q_out overlaps"),
    (dict(), dict(q_out=FAKE + 3 * G, q_row=1536, q_out_row=1536, v_row=1536, v=FAKE + 3 * G - 768), "q_out overlaps"),
    (dict(), dict(q_out=FAKE + 3 * G, q_row=384, q_out_row=384), "q_out"),
])
def test_append_refuses_outputs_over_other_tensors(L, ckw, kw, msg):
    r = L.vdx_rope3d_append(ctypes.byref(_cache(**ckw)), ctypes.byref(_append(**kw)), None)
    assert r == B.VDX_ERR_ARG and msg in L.vdx_last_error().decode(), L.vdx_last_error()


def test_null_structures(L):
    assert L.vdx_rope3d_append(None, ctypes.byref(_append()), None) == B.VDX_ERR_ARG
    assert L.vdx_rope3d_append(ctypes.byref(_cache()), None, None) == B.VDX_ERR_ARG
    assert L.vdx_paged_attn(None, ctypes.byref(_paged()), None) == B.VDX_ERR_ARG
    assert L.vdx_paged_attn(ctypes.byref(_cache()), None, None) == B.VDX_ERR_ARG
    assert L.vdx_cross_attn(None, None) == B.VDX_ERR_ARG


def test_nothing_to_do_launches_nothing(L):
    # no rows, no sequences, no batch: fine without any address
    assert L.vdx_rope3d_append(ctypes.byref(_cache()), ctypes.byref(_append(rows=0)), None) == B.VDX_OK
    assert L.vdx_rope3d_append(ctypes.byref(_cache(seqs=0, page_table=0)), ctypes.byref(_append()), None) == B.VDX_OK
    assert L.vdx_paged_attn(ctypes.byref(_cache()), ctypes.byref(_paged(rows=0, q=0, out=0, lse=0, cu=0)), None) == B.VDX_OK
    assert L.vdx_cross_attn(ctypes.byref(_cross(B=0)), None) == B.VDX_OK
    assert L.vdx_cross_attn(ctypes.byref(_cross(N=0, q=0, out=0, lse=0)), None) == B.VDX_OK


def test_a_workspace_is_asked_for_and_checked(L):
    # long caches of few heads are split along the keys; the partial results need room
    c = _cache(page_size=128, max_pages=512, table_stride=512, num_pages=600, k_page=128 * 512, v_page=128 * 512)
    a = _paged(rows=3, max_q=1)
    need = L.vdx_paged_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(a))
    assert need > 0
    for kw, status, msg in ((dict(), B.VDX_ERR_ARG, "workspace"),
                            (dict(workspace=FAKE + 9 * G, workspace_bytes=need - 1), B.VDX_ERR_ARG, "workspace"),
                            (dict(workspace=FAKE + 9 * G + 8, workspace_bytes=need), B.VDX_ERR_ALIGN, "workspace"),
                            (dict(workspace=FAKE + 4 * G + 16, workspace_bytes=need), B.VDX_ERR_ARG, "workspace overlaps"),
                            (dict(workspace=FAKE + 5 * G, workspace_bytes=need), B.VDX_ERR_ARG, "workspace overlaps")):
        a = _paged(rows=3, max_q=1, **kw)
        assert L.vdx_paged_attn(ctypes.byref(c), ctypes.byref(a), None) == status
        assert msg in L.vdx_last_error().decode()


def test_structures_match_the_header(tmp_path):
    # offsets of every field, as the C compiler lays them out
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "vdx.h"', 'int main(void) {']
    pairs = {"vdx_paged_kv": B.PagedKvStruct, "vdx_append_args": B.AppendArgs, "vdx_paged_attn_args": B.PagedAttnArgs,
             "vdx_cross_attn_args": B.CrossAttnArgs, "vdx_attn_options": B.AttnOptions}
    for name, st in pairs.items():
        src.append(f'printf("{name} %zu\\n", sizeof({name}));')
        for f in st._fields_:
            src.append(f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));')
    src.append("return 0; }")
    (tmp_path / "o.c").write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines())
    hdr = open(os.path.join(ROOT, "include", "vdx.h")).read()
    for name, st in pairs.items():
        assert int(got[name]) == ctypes.sizeof(st)
        for f in st._fields_:
            assert int(got[f"{name}.{f[0]}"]) == getattr(st, f[0]).offset
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), hdr, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        names = [re.sub(r".*[\s*]", "", x.strip()) for decl in body.split(";") for x in decl.split(",") if x.strip()]
        assert names == [f[0] for f in st._fields_]


def test_the_compiled_entry_is_bound_to_its_torch(L, monkeypatch):
    import torch
    from video_diffusion_transformer_rope_gb300 import streaming
    t = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(streaming, "_native", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="build them again"):
        vdx.cross_attn(t, t, t)
    monkeypatch.undo()
    with pytest.raises(vdx.VdxError, match="CUDA tensor"):
        vdx.cross_attn(t, t, t)
    assert not _build._ext_stale(_build._torch()) and _build._ext_stale((os.path.dirname(torch.__file__), "1.0.0"))


def test_python_refuses_host_tensors_and_gradients():
    import torch
    t = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(vdx.VdxError):
        vdx.cross_attn(t, t, t)
    with pytest.raises(vdx.VdxError):
        vdx.rope3d_append(t[0], t[0], t[0], vdx.PagedKV(t, t, torch.zeros(1, 1, dtype=torch.int32)), None, None, (1, 1, 1))
    with pytest.raises(vdx.VdxError):
        vdx.paged_attn(t[0], vdx.PagedKV(t, t, torch.zeros(1, 1, dtype=torch.int32)), None, None)
