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


_torch = None
_raw_stream = None
_I32_MAX = 0x7fffffff


def _t():
    """torch, imported on first use (the library itself loads without it)."""
    global _torch, _raw_stream
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _torch = torch
    return _torch


def _dtype(t):
    torch = _t()
    if t.dtype == torch.bfloat16:
        return B.DTYPE_BF16
    if t.dtype == torch.float16:
        return B.DTYPE_FP16
    raise VdxError(VDX_ERR_UNSUPPORTED, f"dtype {t.dtype} (use bfloat16 or float16)")


def _tensor(name, t, like, dims):
    """A CUDA tensor of `dims` dimensions on like's device with like's dtype and dense channels; its
    shape and strides.  (The checks of these calls are host time of every launch: cheap ones first,
    each attribute once.)"""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda or t.get_device() != like.get_device() or t.dtype != like.dtype:
        raise VdxError(VDX_ERR_ARG, f"{name} must be a CUDA tensor of dtype {like.dtype} on {like.device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != dims:
        raise VdxError(VDX_ERR_ARG, f"{name} must have {dims} dimensions, got {tuple(shape)}")
    if max(shape) > _I32_MAX:
        raise VdxError(VDX_ERR_ARG, f"{name}: {tuple(shape)} is too large")
    if stride[-1] != 1 and shape[-1] > 1:
        raise VdxError(VDX_ERR_ARG, f"{name}: the channels of a head must be contiguous")
    if t.requires_grad and _torch.is_grad_enabled():
        raise VdxError(VDX_ERR_UNSUPPORTED, f"{name} requires a gradient: these calls are forward only "
                                            "(use torch.no_grad() or detach())")
    return shape, stride


def _cuda(name, t):
    torch = _t()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise VdxError(VDX_ERR_ARG, f"{name} must be a CUDA tensor")


def _int32(name, t, like, length):
    if t is None:
        return 0
    if (not isinstance(t, _torch.Tensor) or t.dtype != _torch.int32 or not t.is_cuda or t.get_device() != like.get_device()
            or t.dim() != 1 or t.shape[0] != length or not t.is_contiguous()):
        raise VdxError(VDX_ERR_ARG, f"{name} must be a contiguous int32 CUDA tensor of {length} values on {like.device}")
    return t.data_ptr()


def _ints(name, values, count):
    """`count` integers that fit a C int."""
    values = tuple(map(int, values))
    if len(values) != count or min(values) < 0 or max(values) > _I32_MAX:
        raise VdxError(VDX_ERR_ARG, f"{name} = {values}: {count} integers in [0, 2^31) are needed")
    return values


class _On:
    """The tensors' device and the call's stream, current inside; .handle is the stream."""

    def __init__(self, like, stream):
        if stream.device != like.device:
            raise VdxError(VDX_ERR_ARG, f"the stream is on {stream.device}, the tensors on {like.device}")
        self.handle = stream.cuda_stream
        self.ctx = _torch.cuda.stream(stream)           # also makes the stream's device current

    def __enter__(self):
        self.ctx.__enter__()
        return self.handle

    def __exit__(self, *a):
        return self.ctx.__exit__(*a)


def _run(call, like, stream, *args):
    """call(stream handle, *args) with the tensors' device and the stream current.  Where they are
    already, which is the usual call, nothing is switched: that costs more host time than a launch."""
    if stream is None:
        dev = like.get_device()
        if _torch.cuda.current_device() == dev:
            return call(_raw_stream(dev), *args)
        with _torch.cuda.device(dev):
            return call(_raw_stream(dev), *args)
    with _On(like, stream) as handle:
        return call(handle, *args)


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
        k, v, t = self.k, self.v, self.page_table
        _cuda("the key cache", k)
        ks, kst = _tensor("the key cache", k, k, 4)
        vs, vst = _tensor("the value cache", v, k, 4)
        if ks != vs:
            raise VdxError(VDX_ERR_ARG, f"the key and value caches differ in shape: {tuple(ks)}, {tuple(vs)}")
        torch = _torch
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or t.get_device() != k.get_device()
                or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or max(t.shape) > _I32_MAX):
            raise VdxError(VDX_ERR_ARG, f"page_table must be an int32 [seqs, max_pages] tensor on {k.device} with contiguous rows")
        seqs, width = t.shape
        return B.PagedKvStruct(k.data_ptr(), v.data_ptr(), kst[0], kst[1], kst[2], vst[0], vst[1], vst[2], t.data_ptr(),
                               t.stride(0), ks[0], ks[1], width, ks[2], ks[3], _dtype(k), seqs)


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
    ks, kst = _tensor("k", k, like, 3)
    vs, vst = _tensor("v", v, like, 3)
    rows, d, seqs = ks[0], sc.d, sc.seqs
    if ks[1] != sc.Hkv or ks[2] != d or vs != ks:
        raise VdxError(VDX_ERR_ARG, f"k {tuple(ks)} and v {tuple(vs)} must be [rows, {sc.Hkv}, {d}], as the cache's heads")
    qn = kn = Hq = q_ptr = 0
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and _tensor(name, w, like, 1)[0][0] != d:
            raise VdxError(VDX_ERR_ARG, f"{name} must hold {d} weights")
    if q_norm is not None:
        qn = q_norm.data_ptr()
    if k_norm is not None:
        kn = k_norm.data_ptr()
    qs, qst = None, (0, 0)
    if q is not None:
        qs, qst = _tensor("q", q, like, 3)
        Hq, q_ptr = qs[1], q.data_ptr()
        if qs[0] != rows or qs[2] != d:
            raise VdxError(VDX_ERR_ARG, f"q {tuple(qs)} does not match the {rows} rows of {d} channels of k")
        if Hq == 0:
            raise VdxError(VDX_ERR_ARG, "q has no heads (q=None appends keys and values only)")
        if rows == 0:                                   # empty tensors have no address
            return _torch.empty(qs, dtype=q.dtype, device=q.device) if q_out is None else q_out
    elif q_out is not None:
        raise VdxError(VDX_ERR_ARG, "q_out without q")
    a = B.AppendArgs(q_ptr, k.data_ptr(), v.data_ptr(), 0, qst[0], qst[1], kst[0], kst[1], vst[0], vst[1], 0, 0, rows, Hq,
                     _int32("cu", cu, like, seqs + 1), _int32("kv_len", kv_len, like, seqs),
                     _int32("pos_offset", pos_offset, like, seqs), *_ints("grid", grid, 3), *_ints("sections", sections, 3), theta,
                     qn, kn, eps)
    return _run(_append, like, stream, sc, a, q, qs, q_out)


def _append(handle, sc, a, q, qs, q_out):
    if q is not None:
        if q_out is None:
            q_out = _torch.empty(qs, dtype=q.dtype, device=q.device)
        os_, ost = _tensor("q_out", q_out, q, 3)
        if os_ != qs:
            raise VdxError(VDX_ERR_ARG, f"q_out must be shaped like q {tuple(qs)}")
        a.q_out = q_out.data_ptr()
        a.q_out_row, a.q_out_head = ost[0], ost[1]
    status = B.lib().vdx_rope3d_append(ctypes.byref(sc), ctypes.byref(a), handle)
    if status:
        B._check(status)
    return q_out


def _attention(handle, args, size_fn, run_fn, first, q, lse_shape, out, lse, return_lse, workspace):
    """Outputs and scratch (the caller's, or torch's for this call on its stream), then the call."""
    torch = _torch
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _tensor("out", out, q, q.dim())
        if out.shape != q.shape or not out.is_contiguous():
            raise VdxError(VDX_ERR_ARG, f"out must be contiguous and shaped like q {tuple(q.shape)}")
    args.out = out.data_ptr()
    if lse is not None:
        if (not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or tuple(lse.shape) != lse_shape
                or not lse.is_contiguous() or lse.device != q.device):
            raise VdxError(VDX_ERR_ARG, f"lse must be a contiguous float32 tensor of shape {lse_shape} on {q.device}")
        args.lse = lse.data_ptr()
    elif return_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
        args.lse = lse.data_ptr()
    ref = ctypes.byref(args)
    if workspace is not None:
        if (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.device != q.device
                or not workspace.is_contiguous()):
            raise VdxError(VDX_ERR_ARG, f"workspace must be a contiguous CUDA tensor on {q.device}")
    else:
        need = size_fn(*first, ref)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        args.workspace = workspace.data_ptr()
        args.workspace_bytes = workspace.numel() * workspace.element_size()
    status = run_fn(*first, ref, handle)
    if status:
        B._check(status)
    return out, lse


def _paged_args(q, cache, cu, kv_len, max_q, max_kv, causal_block, scale):
    sc = cache._struct()
    shape, stride = _tensor("q", q, cache.k, 3)
    if shape[2] != sc.d:
        raise VdxError(VDX_ERR_ARG, f"q {tuple(shape)} does not match the cache's head dimension {sc.d}")
    return sc, B.PagedAttnArgs(q.data_ptr(), 0, 0, stride[0], stride[1], shape[0], shape[1],
                               _int32("cu", cu, q, sc.seqs + 1), _int32("kv_len", kv_len, q, sc.seqs),
                               *_ints("max_q, max_kv, causal_block", (max_q or 0, max_kv or 0, causal_block), 3), scale, 0, 0)


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
    sc, a = _paged_args(q, cache, cu, kv_len, max_q, max_kv, causal_block, scale)
    L = B.lib()
    return _run(_attention, q, stream, a, L.vdx_paged_attn_workspace_bytes, L.vdx_paged_attn, (ctypes.byref(sc),), q,
                (a.Hq, a.rows), out, lse, return_lse, workspace)


def paged_attn_workspace_bytes(q, cache, cu, kv_len, max_q=None, max_kv=None):
    """Bytes of scratch that paged_attn needs for these arguments."""
    sc, a = _paged_args(q, cache, cu, kv_len, max_q, max_kv, 0, 0.0)
    with _t().cuda.device(q.device):
        return B.lib().vdx_paged_attn_workspace_bytes(ctypes.byref(sc), ctypes.byref(a))


def _cross_args(q, k, v, kv_len, scale):
    _cuda("q", q)
    qs, qst = _tensor("q", q, q, 4)
    ks, kst = _tensor("k", k, q, 4)
    vs, vst = _tensor("v", v, q, 4)
    if ks != vs or ks[0] != qs[0] or ks[3] != qs[3]:
        raise VdxError(VDX_ERR_ARG, f"q [B, N, Hq, d], k and v [B, M, Hkv, d]: got {tuple(qs)}, {tuple(ks)}, {tuple(vs)}")
    return B.CrossAttnArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, qst[0], qst[1], qst[2], kst[0], kst[1], kst[2],
                           vst[0], vst[1], vst[2], qs[0], qs[1], ks[1], qs[2], ks[2], qs[3], _dtype(q),
                           _int32("kv_len", kv_len, q, qs[0]), scale, 0, 0)


def cross_attn(q, k, v, kv_len=None, scale=0.0, out=None, lse=None, return_lse=True, stream=None, workspace=None):
    """Cross attention: q [B, N, Hq, d] over an encoder's k, v [B, M, Hkv, d] (Hq a multiple of Hkv; no
    positions).  kv_len: optional int32 [B], keys of each batch entry (keys past it may hold anything;
    an entry without keys gives out = 0, lse = -inf).  k, v expanded over the batch are not copied.

    Returns (out [B, N, Hq, d], lse [B, Hq, N] float32 or None)."""
    a = _cross_args(q, k, v, kv_len, scale)
    L = B.lib()
    return _run(_attention, q, stream, a, L.vdx_cross_attn_workspace_bytes, L.vdx_cross_attn, (), q, (a.B, a.Hq, a.N), out,
                lse, return_lse, workspace)


def cross_attn_workspace_bytes(q, k, v, kv_len=None):
    """Bytes of scratch that cross_attn needs for these arguments."""
    a = _cross_args(q, k, v, kv_len, 0.0)
    with _t().cuda.device(q.device):
        return B.lib().vdx_cross_attn_workspace_bytes(ctypes.byref(a))
