"""The vision tower's operators over patch embeddings, on torch tensors:
attention over the plan's chunks with its backward pass.

Argument checks and allocation only: the work runs in the HIP library
(``include/mimo_pre.h``), on the tensors' device and on ``stream`` (default:
torch's current stream there).  Outputs and workspaces that are not passed in
are allocated by torch on that stream.  The framework keeps no autograd
graph: each backward pass is a call of its own.
"""
from __future__ import annotations

import contextlib
import struct

import torch

from . import _abi
from ._abi import MIMO_OK, _require

# mimo_attention and mimo_attention_grads (include/mimo_pre.h)
_ATTENTION = struct.Struct("<q5if2Q" + "Qqq" * 4 + "Q")
_GRADS = struct.Struct("<" + "Qqq" * 4 + "Q")


@contextlib.contextmanager
def _entered(device, stream, tensors):
    index = device.index
    with contextlib.ExitStack() as stack:
        if index != torch.cuda.current_device():
            stack.enter_context(torch.cuda.device(index))
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            stack.enter_context(torch.cuda.stream(stream))
        yield


_NOTHING = contextlib.nullcontext()


def _on(device, stream, tensors, what):
    """The context a call runs in: the tensors' device current, and the
    caller's stream, if one is given, current and known to the allocator as a
    user of the tensors."""
    if stream is not None:
        _require(stream.device == device, lambda: f"{what}: the stream belongs to {stream.device}, the tensors to {device}")
    elif device.index == torch.cuda.current_device():
        return _NOTHING
    return _entered(device, stream, tensors)


def _check(code, what):
    if code != MIMO_OK:
        _abi._check(code, what)


def _heads(t, what, name, shape=None):
    """(pointer, row stride, head stride) of a bf16 [rows, heads, head_dim] tensor."""
    _require(t.dtype == torch.bfloat16 and t.dim() == 3,
             lambda: f"{what}: {name} must be bfloat16 [rows, heads, head_dim], got {tuple(t.shape)} {t.dtype}")
    _require(shape is None or t.shape == shape, lambda: f"{what}: {name} must be {tuple(shape)}, got {tuple(t.shape)}")
    row, head, inner = t.stride()
    rows, heads, dim = t.shape
    _require(inner == 1 or dim == 1, lambda: f"{what}: {name}'s innermost axis must be dense, got strides {t.stride()}")
    # torch leaves the stride of an axis of one free: the library asks for a valid one
    return t.data_ptr(), row if rows > 1 else max(dim, 8), head if heads > 1 else 0


def _vector(t, what, name, n, dtype):
    _require(t.dtype == dtype and t.dim() == 1 and t.shape[0] == n and t.is_contiguous(),
             lambda: f"{what}: {name} must be contiguous {dtype} [{n}], got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _pack_attention(what, q, k, v, cu_seqlens, window, scale, sink, out, lse):
    rows, q_heads, head_dim = q.shape
    _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1 and cu_seqlens.shape[0] >= 1
             and cu_seqlens.is_contiguous(),
             lambda: f"{what}: cu_seqlens must be contiguous int32 [chunks + 1], got {tuple(cu_seqlens.shape)} "
                     f"{cu_seqlens.dtype}")
    if lse is not None:
        _require(lse.dtype == torch.float32 and lse.shape == (q_heads, rows) and lse.is_contiguous(),
                 lambda: f"{what}: lse must be contiguous float32 [{q_heads}, {rows}], got {tuple(lse.shape)} {lse.dtype}")
    if window is None or window < 0:
        window = -1
    return _ATTENTION.pack(
        rows, q_heads, k.shape[1], head_dim, cu_seqlens.shape[0] - 1, min(int(window), 2 ** 31 - 1),
        head_dim ** -0.5 if scale is None else float(scale), cu_seqlens.data_ptr(),
        0 if sink is None else _vector(sink, what, "sink", q_heads, torch.float32),
        *_heads(q, what, "q"), *_heads(k, what, "k"), *_heads(v, what, "v", k.shape),
        *_heads(out, what, "out", q.shape), 0 if lse is None else lse.data_ptr())


def _check_qkv(what, q, k, v):
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _require(t.dim() == 3, lambda: f"{what}: {name} must be [rows, heads, head_dim], got {tuple(t.shape)}")
    rows, q_heads, head_dim = q.shape
    _require(k.shape[0] == rows and k.shape[2] == head_dim and k.shape[1] >= 1 and q_heads >= 1
             and q_heads % k.shape[1] == 0,
             lambda: f"{what}: q {tuple(q.shape)} and k {tuple(k.shape)} must agree in rows and head_dim, and q's heads "
                     "must be a multiple of k's")


def chunk_attention(q, k, v, cu_seqlens, window=-1, scale=None, sink=None, out=None, lse=None,
                    return_lse: bool = False, stream=None):
    """mimo_chunk_attention: attention of every row to the rows of its chunk
    (vision page, MiMoVisionAttention), forward.

    q bf16 [rows, q_heads, head_dim]; k, v bf16 [rows, kv_heads, head_dim],
    each with an innermost axis that is dense and other strides in multiples
    of 8 values (slices of one projection's output are fine); cu_seqlens
    int32 [chunks + 1] on the same GPU (vit_tables' boundaries, moved there
    once).  window >= 0 limits a row to keys at most that far from it in its
    chunk; sink (float32 [q_heads]) is added to each chunk's key 0's logit;
    scale defaults to head_dim ** -0.5.

    Returns out [rows, q_heads, head_dim], or with return_lse=True (out, lse)
    with lse float32 [q_heads, rows], which the backward pass takes.  Rows
    behind cu_seqlens[-1] are left as they were (undefined where out is
    allocated here).
    """
    what = "chunk_attention"
    _check_qkv(what, q, k, v)
    dev = q.device
    with _on(dev, stream, (q, k, v, cu_seqlens, sink, out, lse), what) if dev.type == "cuda" else _NOTHING:
        if dev.type == "cuda":
            if out is None:
                out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
            if lse is None and return_lse:
                lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=dev)
        args = _pack_attention(what, q, k, v, cu_seqlens, window, scale, sink, q if out is None else out, lse)
        _abi._check_device((q, k, v, cu_seqlens, sink, out, lse), what)
        _check(_abi.load().mimo_chunk_attention(args, _abi._stream_handle(stream, dev)), what)
    return (out, lse) if return_lse else out


def chunk_attention_backward(dout, q, k, v, out, lse, cu_seqlens, window=-1, scale=None, sink=None, dq=None, dk=None,
                             dv=None, dsink=None, workspace=None, stream=None):
    """mimo_chunk_attention_backward: the gradients of chunk_attention's
    inputs for dout bf16 [rows, q_heads, head_dim], given its out and lse; the
    probabilities are recomputed.  The other arguments are those of the
    forward call.

    Returns (dq, dk, dv, dsink): bf16 of q's, k's and v's shapes, and float32
    [q_heads], or None without sink.  Gradients are overwritten; rows behind
    cu_seqlens[-1] are left as they were.  ``workspace``: uint8, at least
    chunk_attention_workspace_bytes(rows, q_heads, chunks) bytes; calls that
    may run at the same time need one each.
    """
    what = "chunk_attention_backward"
    _check_qkv(what, q, k, v)
    _require(dsink is None or sink is not None, f"{what}: dsink is given without sink")
    rows, q_heads, _ = q.shape
    dev = q.device
    _require(lse is not None, f"{what}: lse is None (chunk_attention returns it with return_lse=True)")
    ins = (dout, q, k, v, out, lse, cu_seqlens, sink)
    with _on(dev, stream, (*ins, dq, dk, dv, dsink, workspace), what) if dev.type == "cuda" else _NOTHING:
        args = _pack_attention(what, q, k, v, cu_seqlens, window, scale, sink, out, lse)
        dout_heads = _heads(dout, what, "dout", q.shape)
        _abi._check_device(ins, what)
        if dq is None:
            dq = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        if dk is None:
            dk = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
        if dv is None:
            dv = torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
        if dsink is None and sink is not None:
            dsink = torch.empty(q_heads, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(max(chunk_attention_workspace_bytes(rows, q_heads, cu_seqlens.shape[0] - 1), 16),
                                    dtype=torch.uint8, device=dev)
        else:
            _abi._check_bytes(workspace, what + ": workspace")
        grads = _GRADS.pack(*dout_heads, *_heads(dq, what, "dq", q.shape), *_heads(dk, what, "dk", k.shape),
                            *_heads(dv, what, "dv", v.shape),
                            0 if dsink is None else _vector(dsink, what, "dsink", q_heads, torch.float32))
        _abi._check_device((q, dq, dk, dv, dsink, workspace), what)
        _check(_abi.load().mimo_chunk_attention_backward(args, grads, workspace.data_ptr(), workspace.numel(),
                                                         _abi._stream_handle(stream, dev)), what)
    return dq, dk, dv, dsink


def chunk_attention_workspace_bytes(rows: int, q_heads: int, chunks: int) -> int:
    """mimo_chunk_attention_workspace_bytes."""
    return int(_abi.load().mimo_chunk_attention_workspace_bytes(int(rows), int(q_heads), int(chunks)))
