"""Streaming and conditioning calls: appending new tokens to a paged key/value cache, attention of
those tokens over it, and cross attention to an encoder's states (include/vdx.h describes each
operation).  The arguments are marshalled by the compiled module _streaming_py (csrc/streaming_py.cpp),
since these calls are short: no fallback, and every call that the library cannot take raises VdxError
before anything is launched.
"""
import contextlib
import ctypes
from dataclasses import dataclass
from typing import Any

from . import _binding as B
from ._binding import VDX_ERR_ARG, VdxError


_native = None


def _load():
    """The compiled module, bound to libvdx.so, on first use (the library itself loads without torch)."""
    global _native
    import torch
    L = B.lib()
    try:
        from . import _streaming_py as native
    except ImportError as e:
        from . import _build
        why = _build._ext_lacks(_build._torch_base())
        if why:
            raise RuntimeError(f"the streaming calls are not available: {why}") from e
        raise RuntimeError("the compiled entry of the streaming calls is missing or does not load: build it with "
                           f"video_diffusion_transformer_rope_gb300._build.build() ({e})") from e
    if native.TORCH_VERSION.split("+")[0] != torch.__version__.split("+")[0]:
        raise RuntimeError(f"the streaming calls were built for PyTorch {native.TORCH_VERSION}, this is {torch.__version__}: "
                           "build them again with video_diffusion_transformer_rope_gb300._build.build()")
    native.bind(VdxError, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.vdx_rope3d_append, L.vdx_paged_attn_offset, L.vdx_paged_attn_workspace_bytes, L.vdx_cross_attn,
        L.vdx_cross_attn_workspace_bytes, L.vdx_last_error)))
    _native = native
    return native


@contextlib.contextmanager
def _on(stream, like):
    """The stream, and the tensors' device, current inside."""
    import torch
    if not isinstance(like, torch.Tensor) or stream.device != like.device:
        raise VdxError(VDX_ERR_ARG, f"the stream is on {stream.device}, the tensors on {getattr(like, 'device', None)}")
    with torch.cuda.stream(stream):
        yield


@dataclass
class PagedKV:
    """A paged key/value cache: k and v [num_pages, page_size, Hkv, d] (bf16 or fp16 CUDA tensors;
    any token / head order, for example a permuted [num_pages, Hkv, page_size, d]) and page_table
    [seqs, max_pages] int32.  Key c of sequence s is token c % page_size of page
    page_table[s, c // page_size].  page_size: 16, 32, 64 or any size >= 128."""
    k: Any
    v: Any
    page_table: Any


def rope3d_append(q, k, v, cache, cu, kv_len, grid, sections=(0, 0, 0), theta=10000.0, pos_offset=None, q_norm=None,
                  k_norm=None, eps=1e-6, q_out=None, stream=None):
    """Append new tokens to `cache` (a PagedKV): k, v [rows, Hkv, d] go to the cache, k rotated, and
    the rotated q [rows, Hq, d] is returned (in q_out if given; q_out=q rotates in place; q=None
    appends only and returns None).

    cu: int32 [seqs + 1], rows cu[s]:cu[s+1] belong to sequence s; kv_len: int32 [seqs], keys of each
    sequence with the new ones.  grid = (T, Hgrid, Wgrid): the new token with cache index c stands at
    grid token pos_offset[s] + c.  q_norm / k_norm: [d] weights of a per-head RMS norm applied before
    the rotation (a norm over all heads of a token goes before the call).  Slices of a fused projection are taken as they are.  Two rows of a call must not land in
    one slot (a page that two sequences share and both write): it would hold pieces of both."""
    call = (_native or _load()).append
    if stream is None:
        return call(q, k, v, cache.k, cache.v, cache.page_table, cu, kv_len, pos_offset, q_norm, k_norm, eps, q_out, grid,
                    sections, theta)
    with _on(stream, cache.k):
        return call(q, k, v, cache.k, cache.v, cache.page_table, cu, kv_len, pos_offset, q_norm, k_norm, eps, q_out, grid,
                    sections, theta)


def paged_attn(q, cache, cu, kv_len, max_q=None, max_kv=None, causal_block=0, scale=0.0, out=None, lse=None,
               return_lse=True, stream=None, workspace=None, pos_offset=None):
    """Attention of new tokens over the cache: q [rows, Hq, d], already rotated, keys already appended
    (rope3d_append); cu and kv_len as there.  causal_block 0: every row sees all kv_len keys of its
    sequence; 1: the keys up to its own; m: whole blocks of m grid tokens (latent frames) up to its own.
    pos_offset: as in rope3d_append, where a sequence's oldest pages were dropped: blocks are counted from
    grid token 0, so key 0 may stand inside one.

    max_q, max_kv: host bounds on the rows and keys of a sequence (default: rows, and what the page
    table can hold); tight ones make small launches.  workspace: an optional CUDA tensor of
    paged_attn_workspace_bytes(...) bytes (None: taken from torch's allocator).

    Returns (out [rows, Hq, d], lse [Hq, rows] float32 or None); rows outside every sequence are left
    as they were in out / lse."""
    call = (_native or _load()).paged
    if stream is None:
        return call(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv, causal_block, scale, out, lse, return_lse,
                    workspace, pos_offset)
    with _on(stream, q):
        return call(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv, causal_block, scale, out, lse, return_lse,
                    workspace, pos_offset)


def paged_attn_workspace_bytes(q, cache, cu, kv_len, max_q=None, max_kv=None):
    """Bytes of scratch that paged_attn needs for these arguments."""
    return (_native or _load()).paged_size(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv)


def cross_attn(q, k, v, kv_len=None, scale=0.0, out=None, lse=None, return_lse=True, stream=None, workspace=None):
    """Cross attention: q [B, N, Hq, d] over an encoder's k, v [B, M, Hkv, d] (Hq a multiple of Hkv; no
    positions).  kv_len: optional int32 [B], keys of each batch entry (keys past it may hold anything;
    an entry without keys gives out = 0, lse = -inf).  k, v expanded over the batch are not copied.

    Returns (out [B, N, Hq, d], lse [B, Hq, N] float32 or None)."""
    call = (_native or _load()).cross
    if stream is None:
        return call(q, k, v, kv_len, scale, out, lse, return_lse, workspace)
    with _on(stream, q):
        return call(q, k, v, kv_len, scale, out, lse, return_lse, workspace)


def cross_attn_workspace_bytes(q, k, v, kv_len=None):
    """Bytes of scratch that cross_attn needs for these arguments."""
    return (_native or _load()).cross_size(q, k, v, kv_len)
