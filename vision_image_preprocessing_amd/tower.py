"""The vision tower's operators over patch embeddings, on torch tensors:
attention over the plan's chunks and layer norm, each with its backward pass,
and the matrix product in 8-bit integers.

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


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_CODES = {torch.float32: _abi.MIMO_F32, torch.bfloat16: _abi.MIMO_BF16}
_KINDS = (torch.float32, torch.bfloat16)


def _out_type(what, out_dtype, default=None):
    if out_dtype is None and default is not None:
        return default
    _require(out_dtype in _TYPES, lambda: f"{what}: out_dtype {out_dtype!r} is not f32 or bf16")
    return _TYPES[out_dtype]


def _matrix(t, what, name, shape=None, dtypes=_KINDS):
    """A dense [rows, width] tensor of one of dtypes."""
    _require(t.dim() == 2 and t.dtype in dtypes and t.is_contiguous(),
             lambda: f"{what}: {name} must be a contiguous [rows, width] tensor of "
                     f"{' or '.join(str(d) for d in dtypes)}, got {tuple(t.shape)} {t.dtype}"
                     + ("" if t.is_contiguous() else " (not contiguous)"))
    _require(shape is None or t.shape == shape, lambda: f"{what}: {name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _pointer(t):
    return None if t is None else t.data_ptr()


def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, out=None, out_dtype=None, return_stats: bool = False,
               mean=None, rstd=None, stream=None):
    """mimo_layer_norm: (x - mean) * rstd * weight + bias of each row of x
    [rows, width] (float32 or bf16, contiguous; merge units are a view of four
    rows as one); weight and bias float32 [width] or None.

    Returns out [rows, width] of out_dtype ("f32" or "bf16"; x's by default),
    or with return_stats=True (out, mean, rstd) with float32 [rows]
    statistics, which the backward pass takes.  out may be x itself where the
    dtypes agree.
    """
    what = "layer_norm"
    _matrix(x, what, "x")
    rows, width = x.shape
    _require(width >= 1, lambda: f"{what}: x has no columns")
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _vector(t, what, name, width, torch.float32)
    dev = x.device
    dtype = out.dtype if out is not None else _out_type(what, out_dtype, x.dtype)
    if out is not None:
        _matrix(out, what, "out", x.shape)
    _abi._check_device((x, weight, bias, out, mean, rstd), what)
    with _on(dev, stream, (x, weight, bias, out, mean, rstd), what):
        if out is None:
            out = torch.empty((rows, width), dtype=dtype, device=dev)
        if return_stats:
            if mean is None:
                mean = torch.empty(rows, dtype=torch.float32, device=dev)
            if rstd is None:
                rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        for t, name in ((mean, "mean"), (rstd, "rstd")):
            if t is not None:
                _vector(t, what, name, rows, torch.float32)
        _check(_abi.load().mimo_layer_norm(rows, width, x.data_ptr(), _CODES[x.dtype], _pointer(weight), _pointer(bias),
                                           float(eps), _CODES[dtype], out.data_ptr(), _pointer(mean), _pointer(rstd),
                                           _abi._stream_handle(stream, dev)), what)
    return (out, mean, rstd) if return_stats else out


def layer_norm_backward(dout, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, affine=None, workspace=None,
                        stream=None):
    """mimo_layer_norm_backward: the gradients of layer_norm's x, weight and
    bias for dout [rows, width] (float32 or bf16), given x and the forward
    call's mean and rstd.

    Returns (dx, dweight, dbias): x's dtype, and float32 [width] each.  The
    sums over rows are made where weight is given, or with affine=True (a norm
    with a bias alone needs dbias too); otherwise, or with affine=False, those
    two that are not passed in are None.  ``workspace``: uint8, at least
    layer_norm_workspace_bytes(rows, width) bytes; calls that may run at the
    same time need one each.
    """
    what = "layer_norm_backward"
    _matrix(x, what, "x")
    rows, width = x.shape
    _require(width >= 1, lambda: f"{what}: x has no columns")
    _matrix(dout, what, "dout", x.shape)
    for t, name, n in ((mean, "mean", rows), (rstd, "rstd", rows), (weight, "weight", width), (dweight, "dweight", width),
                       (dbias, "dbias", width)):
        if t is not None:
            _vector(t, what, name, n, torch.float32)
    _require(mean is not None and rstd is not None, f"{what}: mean and rstd are needed (layer_norm returns them with return_stats=True)")
    if dx is not None:
        _matrix(dx, what, "dx", x.shape, (x.dtype,))
    dev = x.device
    tensors = (dout, x, mean, rstd, weight, dx, dweight, dbias, workspace)
    _abi._check_device(tensors, what)
    with _on(dev, stream, tensors, what):
        if dx is None:
            dx = torch.empty((rows, width), dtype=x.dtype, device=dev)
        if weight is not None if affine is None else affine:
            if dweight is None:
                dweight = torch.empty(width, dtype=torch.float32, device=dev)
            if dbias is None:
                dbias = torch.empty(width, dtype=torch.float32, device=dev)
        if workspace is not None:
            _abi._check_bytes(workspace, what + ": workspace")
        elif dweight is not None or dbias is not None:
            workspace = torch.empty(max(layer_norm_workspace_bytes(rows, width), 16), dtype=torch.uint8, device=dev)
        _check(_abi.load().mimo_layer_norm_backward(
            rows, width, x.data_ptr(), _CODES[x.dtype], dout.data_ptr(), _CODES[dout.dtype], _pointer(weight),
            mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _pointer(dweight), _pointer(dbias), _pointer(workspace),
            0 if workspace is None else workspace.numel(), _abi._stream_handle(stream, dev)), what)
    return dx, dweight, dbias


def layer_norm_workspace_bytes(rows: int, width: int) -> int:
    """mimo_layer_norm_workspace_bytes."""
    return int(_abi.load().mimo_layer_norm_workspace_bytes(int(rows), int(width)))


def quantize_rows(x, q=None, scale=None, stream=None):
    """mimo_quantize_rows: x [rows, width] (float32 or bf16, contiguous) to
    8-bit integers, row by row: activations, or a weight [out, in] by output
    channels.

    Returns (q, scale): int8 [rows, padded], padded = width rounded up to a
    multiple of 128 (zeros behind width), and float32 [rows]; x is near
    q[:, :width] * scale[:, None].
    """
    what = "quantize_rows"
    _matrix(x, what, "x")
    rows, width = x.shape
    _require(width >= 1, lambda: f"{what}: x has no columns")
    padded = (width + 127) // 128 * 128
    if q is not None:
        _matrix(q, what, "q", (rows, padded), (torch.int8,))
    if scale is not None:
        _vector(scale, what, "scale", rows, torch.float32)
    dev = x.device
    _abi._check_device((x, q, scale), what)
    with _on(dev, stream, (x, q, scale), what):
        if q is None:
            q = torch.empty((rows, padded), dtype=torch.int8, device=dev)
        if scale is None:
            scale = torch.empty(rows, dtype=torch.float32, device=dev)
        _check(_abi.load().mimo_quantize_rows(rows, width, x.data_ptr(), _CODES[x.dtype], q.data_ptr(), scale.data_ptr(),
                                              _abi._stream_handle(stream, dev)), what)
    return q, scale


def quantized_linear(xq, x_scale, wq, w_scale, bias=None, out=None, out_dtype: str = "bf16", stream=None):
    """mimo_quantized_linear: (xq @ wq.T) * x_scale[:, None] * w_scale + bias,
    the product in 8-bit integers with exact sums.

    xq int8 [rows, k] and x_scale float32 [rows], wq int8 [out, k] and w_scale
    float32 [out]: quantize_rows' outputs of the activations and the weight (k
    is its padded width); bias float32 [out] or None.  Returns out [rows, out]
    of out_dtype ("f32" or "bf16").
    """
    what = "quantized_linear"
    _matrix(xq, what, "xq", dtypes=(torch.int8,))
    _matrix(wq, what, "wq", dtypes=(torch.int8,))
    rows, k = xq.shape
    n = wq.shape[0]
    _require(wq.shape[1] == k and k >= 128 and k % 128 == 0 and n >= 1,
             lambda: f"{what}: xq {tuple(xq.shape)} and wq {tuple(wq.shape)} must share a width that is a multiple of 128")
    _vector(x_scale, what, "x_scale", rows, torch.float32)
    _vector(w_scale, what, "w_scale", n, torch.float32)
    if bias is not None:
        _vector(bias, what, "bias", n, torch.float32)
    dtype = out.dtype if out is not None else _out_type(what, out_dtype)
    if out is not None:
        _matrix(out, what, "out", (rows, n))
    dev = xq.device
    tensors = (xq, x_scale, wq, w_scale, bias, out)
    _abi._check_device(tensors, what)
    with _on(dev, stream, tensors, what):
        if out is None:
            out = torch.empty((rows, n), dtype=dtype, device=dev)
        _check(_abi.load().mimo_quantized_linear(rows, k, xq.data_ptr(), x_scale.data_ptr(), n, wq.data_ptr(),
                                                 w_scale.data_ptr(), _pointer(bias), _CODES[dtype], out.data_ptr(),
                                                 _abi._stream_handle(stream, dev)), what)
    return out
