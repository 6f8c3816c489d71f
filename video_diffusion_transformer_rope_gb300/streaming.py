"""Streaming and conditioning calls: appending new tokens to a paged key/value cache (of 16 or 8 bits), attention of
those tokens over it, the weight that its keys gather and their eviction, and cross attention to an encoder's
states (include/vdx.h describes each operation).  The arguments are marshalled by the compiled module _streaming_py (csrc/streaming_py.cpp),
since these calls are short: no fallback, and every call that the library cannot take raises VdxError
before anything is launched.
"""
import collections
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
        L.vdx_cross_attn_workspace_bytes, L.vdx_rope3d_append8, L.vdx_paged_attn8, L.vdx_paged_attn8_workspace_bytes,
        L.vdx_paged_attn_weights, L.vdx_paged_evict, L.vdx_last_error)))
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
    page_table[s, c // page_size].  page_size: 16, 32, 64 or any size >= 128.

    In 8 bits k and v are float8_e4m3fn, and k_scale, v_scale [num_pages, ceil(page_size / 16), Hkv]
    float8_e8m0fnu: a power of two for every KV8_BLOCK = 16 tokens of a page and head, which their codes are
    multiplied by.  The other tensors of a call over such a cache are bf16 or fp16, whichever they are."""
    k: Any
    v: Any
    page_table: Any
    k_scale: Any = None
    v_scale: Any = None


KV8_BLOCK = 16
Evicted = collections.namedtuple("Evicted", ["kv_len", "pos_offset", "weights", "index"])


def rope3d_append(q, k, v, cache, cu, kv_len, grid, sections=(0, 0, 0), theta=10000.0, pos_offset=None, q_norm=None,
                  k_norm=None, eps=1e-6, q_out=None, stream=None):
    """Append new tokens to `cache` (a PagedKV): k, v [rows, Hkv, d] go to the cache, k rotated, and
    the rotated q [rows, Hq, d] is returned (in q_out if given; q_out=q rotates in place; q=None
    appends only and returns None).

    cu: int32 [seqs + 1], rows cu[s]:cu[s+1] belong to sequence s; kv_len: int32 [seqs], keys of each
    sequence with the new ones.  grid = (T, Hgrid, Wgrid): the new token with cache index c stands at
    grid token pos_offset[s] + c.  q_norm / k_norm: [d] weights of a per-head RMS norm applied before
    the rotation (a norm over all heads of a token goes before the call).  Slices of a fused projection are taken as they are.  Two rows of a call must not land in
    one slot (a page that two sequences share and both write): it would hold pieces of both.

    An 8-bit cache gets codes of the fp32 keys and values and the scales of the blocks that they land in (a scale grows
    where new values need it, and the block's older codes are rounded again); sync_check() reports values past
    448 * 2^7, which are clamped.  Two sequences must not append into one block of such a cache."""
    call = (_native or _load()).append
    if stream is None:
        return call(q, k, v, cache.k, cache.v, cache.page_table, cu, kv_len, pos_offset, q_norm, k_norm, eps, q_out, grid,
                    sections, theta, cache.k_scale, cache.v_scale)
    with _on(stream, cache.k):
        return call(q, k, v, cache.k, cache.v, cache.page_table, cu, kv_len, pos_offset, q_norm, k_norm, eps, q_out, grid,
                    sections, theta, cache.k_scale, cache.v_scale)


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
                    workspace, pos_offset, cache.k_scale, cache.v_scale)
    with _on(stream, q):
        return call(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv, causal_block, scale, out, lse, return_lse,
                    workspace, pos_offset, cache.k_scale, cache.v_scale)


def paged_attn_workspace_bytes(q, cache, cu, kv_len, max_q=None, max_kv=None):
    """Bytes of scratch that paged_attn needs for these arguments."""
    return (_native or _load()).paged_size(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv, cache.k_scale,
                                               cache.v_scale)


def paged_attn_weights(q, cache, cu, kv_len, lse, weights, max_q=None, max_kv=None, causal_block=0, scale=0.0, decay=1.0,
                       pos_offset=None, stream=None):
    """Add up, key by key, what the rows of a paged_attn call weighed: weights float32 [seqs, Hkv, width], in place (and
    returned).  Arguments as in that call, with the lse [Hq, rows] that it returned.  For each sequence with rows,

        weights[s, h, c] = decay * weights[s, h, c] + sum over rows and query heads of group h of exp(score - lse)

    for its keys c, those of the call's own rows starting from 0, so the buffer needs no clearing.  Keys that a row does
    not see get nothing from it; entries past a sequence's keys, and sequences without rows, stay as they are."""
    call = (_native or _load()).weights
    if stream is None:
        return call(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv, lse, weights, causal_block, scale, decay,
                    pos_offset, cache.k_scale, cache.v_scale)
    with _on(stream, q):
        return call(q, cache.k, cache.v, cache.page_table, cu, kv_len, max_q, max_kv, lse, weights, causal_block, scale, decay,
                    pos_offset, cache.k_scale, cache.v_scale)


def paged_evict(cache, weights, kv_len, keep, into, recent=0, max_kv=None, pos_offset=None, weights_out=None, stream=None):
    """Evict from `cache` the keys that gathered least, for each sequence and kv head: of more than `keep` keys the last
    `recent` stay and, of the others, the keep - recent with the largest weights (of equals the first); of fewer, all.
    What stays moves, in order, to cache indices 0, 1, .. of `into`: a PagedKV of the same kind with another page
    table, in the same pools or others, whose pages the call must not read too.  Afterwards the old pages are free.

    weights: float32 [seqs, Hkv, width], from paged_attn_weights (float("inf") pins a key, NaN counts as the largest).
    Returns Evicted(kv_len, pos_offset, weights, index): the new lengths; the position offsets with which the next
    tokens are appended and attend (pos_offset, or 0, and what each sequence lost); the weights of what stayed and
    the old cache indices of it, [seqs, Hkv, keep] with 0 and -1 past the new lengths.  weights_out: a buffer for the
    weights, at least keep wide; it may be `weights` itself."""
    call = (_native or _load()).evict
    if stream is None:
        return Evicted(*call(cache.k, cache.v, cache.page_table, cache.k_scale, cache.v_scale, weights, kv_len, keep, recent, max_kv,
                             pos_offset, weights_out, into.k, into.v, into.page_table, into.k_scale, into.v_scale))
    with _on(stream, cache.k):
        return Evicted(*call(cache.k, cache.v, cache.page_table, cache.k_scale, cache.v_scale, weights, kv_len, keep, recent, max_kv,
                             pos_offset, weights_out, into.k, into.v, into.page_table, into.k_scale, into.v_scale))


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
