"""Streaming and conditioning calls: appending new tokens to a paged key/value cache, attention of
those tokens over it, and cross attention to an encoder's states (include/vdx.h describes each
operation).  Argument marshalling only, as in _binding.py: no fallback, and every call that the
library cannot take raises VdxError before anything is launched.
"""
import ctypes
from dataclasses import dataclass
from typing import Any

from . import _binding as B
from ._binding import VDX_ERR_ARG, VDX_ERR_UNSUPPORTED, VdxError


def _dtype(t):
    import torch
    if t.dtype == torch.bfloat16:
        return B.DTYPE_BF16
    if t.dtype == torch.float16:
        return B.DTYPE_FP16
    raise VdxError(VDX_ERR_UNSUPPORTED, f"dtype {t.dtype} (use bfloat16 or float16)")


def _tensor(name, t, like, dims, writable=False):
    """A CUDA tensor of `dims` dimensions on like's device with like's dtype and dense channels."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != like.device or t.dtype != like.dtype:
        raise VdxError(VDX_ERR_ARG, f"{name} must be a CUDA tensor of dtype {like.dtype} on {like.device}")
    if t.dim() != dims:
        raise VdxError(VDX_ERR_ARG, f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise VdxError(VDX_ERR_ARG, f"{name}: the channels of a head must be contiguous")
    if t.requires_grad and torch.is_grad_enabled():
        raise VdxError(VDX_ERR_UNSUPPORTED, f"{name} requires a gradient: these calls are forward only "
                                            "(use torch.no_grad() or detach())")


def _int32(name, t, like, length):
    import torch
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != like.device or t.dtype != torch.int32
            or t.dim() != 1 or t.shape[0] != length or (length > 1 and t.stride(0) != 1)):
        raise VdxError(VDX_ERR_ARG, f"{name} must be a contiguous int32 CUDA tensor of {length} values on {like.device}")
    return t.data_ptr()


def _int(name, x, least=0):
    x = int(x)
    if x < least or x > 0x7fffffff:
        raise VdxError(VDX_ERR_ARG, f"{name} = {x} is outside [{least}, 2^31)")
    return x


class _On:
    """The tensors' device and the call's stream are current inside; .handle is the stream."""

    def __init__(self, like, stream):
        import torch
        self.stream = torch.cuda.current_stream(like.device) if stream is None else stream
        if self.stream.device != like.device:
            raise VdxError(VDX_ERR_ARG, f"the stream is on {self.stream.device}, the tensors on {like.device}")
        self.ctx = torch.cuda.stream(self.stream)       # also makes the stream's device current
        self.handle = ctypes.c_void_p(self.stream.cuda_stream)

    def __enter__(self):
        self.ctx.__enter__()
        return self

    def __exit__(self, *a):
        return self.ctx.__exit__(*a)


@dataclass
class PagedKV:
    """A paged key/value cache: k and v [num_pages, page_size, Hkv, d] (bf16 or fp16 CUDA tensors;
    any token / head order, for example a permuted [num_pages, Hkv, page_size, d]) and page_table
    [seqs, max_pages] int32.  Key c of sequence s is token c % page_size of page
    page_table[s, c // page_size].  page_size: 16, 32, 64 or any size >= 128."""
    k: Any
    v: Any
    page_table: Any

    def _struct(self):
        import torch
        k, v, t = self.k, self.v, self.page_table
        if not isinstance(k, torch.Tensor) or not k.is_cuda:
            raise VdxError(VDX_ERR_ARG, "the key cache must be a CUDA tensor")
        _tensor("the key cache", k, k, 4)
        _tensor("the value cache", v, k, 4)
        if k.shape != v.shape:
            raise VdxError(VDX_ERR_ARG, f"the key and value caches differ in shape: {tuple(k.shape)}, {tuple(v.shape)}")
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != k.device or t.dim() != 2
                or (t.shape[1] > 1 and t.stride(1) != 1)):
            raise VdxError(VDX_ERR_ARG, f"page_table must be an int32 [seqs, max_pages] tensor on {k.device} with contiguous rows")
        return B.PagedKvStruct(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), v.stride(0), v.stride(1),
                               v.stride(2), t.data_ptr(), t.stride(0), k.shape[0], k.shape[1], t.shape[1], k.shape[2],
                               k.shape[3], _dtype(k), t.shape[0])


def rope3d_append(q, k, v, cache, cu, kv_len, grid, sections=(0, 0, 0), theta=10000.0, pos_offset=None, q_norm=None,
                  k_norm=None, eps=1e-6, q_out=None, stream=None):
    """Append new tokens to `cache` (a PagedKV): k, v [rows, Hkv, d] go to the cache, k rotated, and
    the rotated q [rows, Hq, d] is returned (in q_out if given; q_out=q rotates in place; q=None
    appends only and returns None).

    cu: int32 [seqs + 1], rows cu[s]:cu[s+1] belong to sequence s; kv_len: int32 [seqs], keys of each
    sequence with the new ones.  grid = (T, Hgrid, Wgrid): the new token with cache index c stands at
    grid token pos_offset[s] + c.  q_norm / k_norm: [d] weights of a per-head RMS norm applied before
    the rotation.  Slices of a fused projection are taken as they are."""
    sc = cache._struct()
    like = cache.k
    for name, t, h in (("q", q, None), ("k", k, sc.Hkv), ("v", v, sc.Hkv)):
        if t is None and name == "q":
            continue
        _tensor(name, t, like, 3)
        if t.shape[0] != k.shape[0] or t.shape[2] != sc.d or (h is not None and t.shape[1] != h):
            raise VdxError(VDX_ERR_ARG, f"{name} {tuple(t.shape)} does not match [rows, heads, d] of k {tuple(k.shape)} and "
                                        f"the cache's {sc.Hkv} heads of {sc.d}")
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None:
            _tensor(name, w, like, 1)
            if w.shape[0] != sc.d:
                raise VdxError(VDX_ERR_ARG, f"{name} must hold {sc.d} weights")
    T, Hg, Wg = (_int("grid", x) for x in grid)
    st, sh, sw = (_int("sections", x) for x in sections)
    with _On(like, stream) as on:
        import torch
        if q is None:
            if q_out is not None:
                raise VdxError(VDX_ERR_ARG, "q_out without q")
        elif q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            _tensor("q_out", q_out, like, 3)
            if q_out.shape != q.shape:
                raise VdxError(VDX_ERR_ARG, f"q_out must be shaped like q {tuple(q.shape)}")
        qs = (q.stride(0), q.stride(1)) if q is not None else (0, 0)
        os_ = (q_out.stride(0), q_out.stride(1)) if q is not None else (0, 0)
        a = B.AppendArgs(q.data_ptr() if q is not None else 0, k.data_ptr(), v.data_ptr(),
                         q_out.data_ptr() if q is not None else 0, *qs, k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                         *os_, k.shape[0], q.shape[1] if q is not None else 0, _int32("cu", cu, like, sc.seqs + 1),
                         _int32("kv_len", kv_len, like, sc.seqs), _int32("pos_offset", pos_offset, like, sc.seqs), T, Hg, Wg,
                         st, sh, sw, float(theta), q_norm.data_ptr() if q_norm is not None else 0,
                         k_norm.data_ptr() if k_norm is not None else 0, float(eps))
        if q is not None and q.numel() == 0:            # no rows: empty tensors have no address
            return q_out
        B._check(B.lib().vdx_rope3d_append(ctypes.byref(sc), ctypes.byref(a), on.handle))
    return q_out


def _outputs(q, lse_shape, out, lse, return_lse):
    import torch
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _tensor("out", out, q, q.dim())
        if out.shape != q.shape or not out.is_contiguous():
            raise VdxError(VDX_ERR_ARG, f"out must be contiguous and shaped like q {tuple(q.shape)}")
    if lse is None:
        if return_lse:
            lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    elif (lse.dtype != torch.float32 or tuple(lse.shape) != tuple(lse_shape) or not lse.is_contiguous()
          or lse.device != q.device):
        raise VdxError(VDX_ERR_ARG, f"lse must be a contiguous float32 tensor of shape {tuple(lse_shape)} on {q.device}")
    return out, lse


def _with_workspace(args, size_fn, run_fn, workspace, like, on):
    """Fill args.workspace (the caller's tensor, or one taken from torch's allocator for this call on
    its stream) and run."""
    import torch
    if workspace is not None:
        if (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.device != like.device
                or not workspace.is_contiguous()):
            raise VdxError(VDX_ERR_ARG, f"workspace must be a contiguous CUDA tensor on {like.device}")
    else:
        need = size_fn()
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    if workspace is not None:
        args.workspace = workspace.data_ptr()
        args.workspace_bytes = workspace.numel() * workspace.element_size()
    B._check(run_fn(on.handle))


def _paged_args(q, sc, cu, kv_len, max_q, max_kv, causal_block, scale):
    return B.PagedAttnArgs(q.data_ptr(), 0, 0, q.stride(0), q.stride(1), q.shape[0], q.shape[1],
                           _int32("cu", cu, q, sc.seqs + 1), _int32("kv_len", kv_len, q, sc.seqs), _int("max_q", max_q or 0),
                           _int("max_kv", max_kv or 0), _int("causal_block", causal_block), float(scale), 0, 0)


def paged_attn(q, cache, cu, kv_len, max_q=None, max_kv=None, causal_block=0, scale=0.0, out=None, lse=None,
               return_lse=True, stream=None, workspace=None):
    """Attention of new tokens over the cache: q [rows, Hq, d], already rotated, keys already appended
    (rope3d_append); cu and kv_len as there.  causal_block 0: every row sees all kv_len keys of its
    sequence; 1: the keys up to its own; m: whole blocks of m keys (latent frames) up to its own.

    max_q, max_kv: host bounds on the rows and keys of a sequence (default: rows, and what the page
    table can hold); tight ones make small launches.  workspace: an optional CUDA tensor of
    paged_attn_workspace_bytes(...) bytes (None: taken from torch's allocator).

    Returns (out [rows, Hq, d], lse [Hq, rows] float32 or None); rows outside every sequence are left
    as they were in out / lse."""
    sc = cache._struct()
    _tensor("q", q, cache.k, 3)
    if q.shape[2] != sc.d:
        raise VdxError(VDX_ERR_ARG, f"q {tuple(q.shape)} does not match the cache's head dimension {sc.d}")
    a = _paged_args(q, sc, cu, kv_len, max_q, max_kv, causal_block, scale)
    L = B.lib()
    with _On(q, stream) as on:
        out, lse = _outputs(q, (q.shape[1], q.shape[0]), out, lse, return_lse)
        a.out, a.lse = out.data_ptr(), lse.data_ptr() if lse is not None else 0
        _with_workspace(a, lambda: L.vdx_paged_attn_workspace_bytes(ctypes.byref(sc), ctypes.byref(a)),
                        lambda h: L.vdx_paged_attn(ctypes.byref(sc), ctypes.byref(a), h), workspace, q, on)
    return out, lse


def paged_attn_workspace_bytes(q, cache, cu, kv_len, max_q=None, max_kv=None):
    """Bytes of scratch that paged_attn needs for these arguments."""
    import torch
    sc = cache._struct()
    a = _paged_args(q, sc, cu, kv_len, max_q, max_kv, 0, 0.0)
    with torch.cuda.device(q.device):
        return B.lib().vdx_paged_attn_workspace_bytes(ctypes.byref(sc), ctypes.byref(a))


def _cross_args(q, k, v, kv_len, scale):
    import torch
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise VdxError(VDX_ERR_ARG, "q must be a CUDA tensor")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _tensor(name, t, q, 4)
    Bn, N, Hq, d = q.shape
    if k.shape != v.shape or k.shape[0] != Bn or k.shape[3] != d:
        raise VdxError(VDX_ERR_ARG, f"q [B, N, Hq, d], k and v [B, M, Hkv, d]: got {tuple(q.shape)}, {tuple(k.shape)}, "
                                    f"{tuple(v.shape)}")
    return B.CrossAttnArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, *q.stride()[:3], *k.stride()[:3],
                           *v.stride()[:3], Bn, N, k.shape[1], Hq, k.shape[2], d, _dtype(q),
                           _int32("kv_len", kv_len, q, Bn), float(scale), 0, 0)


def cross_attn(q, k, v, kv_len=None, scale=0.0, out=None, lse=None, return_lse=True, stream=None, workspace=None):
    """Cross attention: q [B, N, Hq, d] over an encoder's k, v [B, M, Hkv, d] (Hq a multiple of Hkv; no
    positions).  kv_len: optional int32 [B], keys of each batch entry (keys past it may hold anything;
    an entry without keys gives out = 0, lse = -inf).  k, v expanded over the batch are not copied.

    Returns (out [B, N, Hq, d], lse [B, Hq, N] float32 or None)."""
    a = _cross_args(q, k, v, kv_len, scale)
    L = B.lib()
    with _On(q, stream) as on:
        out, lse = _outputs(q, (q.shape[0], q.shape[2], q.shape[1]), out, lse, return_lse)
        a.out, a.lse = out.data_ptr(), lse.data_ptr() if lse is not None else 0
        _with_workspace(a, lambda: L.vdx_cross_attn_workspace_bytes(ctypes.byref(a)),
                        lambda h: L.vdx_cross_attn(ctypes.byref(a), h), workspace, q, on)
    return out, lse


def cross_attn_workspace_bytes(q, k, v, kv_len=None):
    """Bytes of scratch that cross_attn needs for these arguments."""
    import torch
    a = _cross_args(q, k, v, kv_len, 0.0)
    with torch.cuda.device(q.device):
        return B.lib().vdx_cross_attn_workspace_bytes(ctypes.byref(a))
