"""The vision tower's operators over patch embeddings, on torch tensors:
attention over the plan's chunks and layer norm, each with its backward pass,
and the matrix product in 8-bit integers.

Argument checks and allocation only: the work runs in the HIP library
(``include/mimo_pre.h``), on the tensors' device and on ``stream`` (default:
torch's current stream there).  Outputs and workspaces that are not passed in
are allocated by torch on that stream.  The framework keeps no autograd
graph: each backward pass is a call of its own.

A small call is bound by the host, so the checks are written to cost a few
hundred nanoseconds: attributes compared in place, messages formed on failure
only (one small image's norm, issued back to back: 5.9 us a call, against 10.7
with a message closure and a device object for every check).
"""
from __future__ import annotations

import contextlib
import struct

import torch

from . import _abi
from ._abi import MIMO_BF16, MIMO_E_INVALID, MIMO_E_TOO_LARGE, MIMO_F32, MimoError

_F32, _BF16, _I8, _I32 = torch.float32, torch.bfloat16, torch.int8, torch.int32
_TYPES = {"f32": _F32, "bf16": _BF16}
_CODES = {_F32: MIMO_F32, _BF16: MIMO_BF16}
_device_now = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)

# mimo_attention and mimo_attention_grads (include/mimo_pre.h)
_ATTENTION = struct.Struct("<q5if2Q" + "Qqq" * 4 + "Q")
_GRADS = struct.Struct("<" + "Qqq" * 4 + "Q")

_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = _abi.load()
    return _lib


def _refuse(message):
    raise MimoError(MIMO_E_INVALID, message)


def _refuse_size(message):
    """The library's size limits, looked at before outputs are allocated: those
    of a call that it would refuse might not fit the card."""
    raise MimoError(MIMO_E_TOO_LARGE, message)


def _check_devices(what, tensors):
    """Refuses tensors that are not all on one GPU, as the binding does."""
    _abi._check_device(tensors, what)
    _refuse(f"{what}: every tensor must be on one GPU")  # not reached: the callers have seen a difference


@contextlib.contextmanager
def _entered(what, index, stream, tensors):
    """The context of a call that is not where torch is: the tensors' device
    made current, and the caller's stream, if one is given, current and known
    to the allocator as a user of the tensors.  The entry points call
    themselves again inside it, without the stream."""
    if stream is not None and stream.device.index != index:
        _refuse(f"{what}: the stream belongs to {stream.device}, the tensors to cuda:{index}")
    with torch.cuda.device(index), contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        yield


def _check_vector(what, name, t, n, dtype):
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        _refuse(f"{what}: {name} must be contiguous {dtype} [{n}], got {tuple(t.shape)} {t.dtype}")


def _check_matrix(what, name, t, dtypes=_CODES):
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_contiguous():
        _refuse(f"{what}: {name} must be a contiguous [rows, width] tensor of {' or '.join(str(d) for d in dtypes)}, "
                f"got {tuple(t.shape)} {t.dtype}" + ("" if t.is_contiguous() else " (not contiguous)"))


def _check_shape(what, name, t, shape):
    if t.shape != shape:
        _refuse(f"{what}: {name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _pointer(t):
    return None if t is None else t.data_ptr()


def _dense_like(t):
    """An uninitialised dense tensor of t's shape, type and device (the quickest of torch's ways)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


# ------------------------------------------------------------------ attention

def _heads(what, name, t, shape):
    """(pointer, row stride, head stride) of a bf16 [rows, heads, head_dim] tensor."""
    rows, heads, dim = shape
    if t.dtype is not _BF16 or t.shape != shape:
        _refuse(f"{what}: {name} must be bfloat16 {tuple(shape)} ([rows, heads, head_dim]), got {tuple(t.shape)} {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), heads * dim, dim
    row, head, inner = t.stride()
    if inner != 1 and dim != 1:
        _refuse(f"{what}: {name}'s innermost axis must be dense, got strides {t.stride()}")
    # torch leaves the stride of an axis of one free: the library asks for a valid one
    return t.data_ptr(), row if rows > 1 else max(dim, 8), head if heads > 1 else 0


def _check_qkv(what, q, k, v, cu_seqlens, sink, lse):
    if q.dim() != 3 or k.dim() != 3:
        _refuse(f"{what}: {'q' if q.dim() != 3 else 'k'} must be [rows, heads, head_dim], got "
                f"{tuple(q.shape if q.dim() != 3 else k.shape)}")
    rows, q_heads, head_dim = q.shape
    krows, kv_heads, kdim = k.shape
    if krows != rows or kdim != head_dim or kv_heads < 1 or q_heads < 1 or q_heads % kv_heads:
        _refuse(f"{what}: q {tuple(q.shape)} and k {tuple(k.shape)} must agree in rows and head_dim, and q's heads must be a "
                "multiple of k's")
    if v.shape != k.shape:
        _refuse(f"{what}: v must be of k's shape {tuple(k.shape)}, got {tuple(v.shape)}")
    if cu_seqlens.dtype != _I32 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or not cu_seqlens.is_contiguous():
        _refuse(f"{what}: cu_seqlens must be contiguous int32 [chunks + 1], got {tuple(cu_seqlens.shape)} {cu_seqlens.dtype}")
    chunks = cu_seqlens.shape[0] - 1
    if rows > 0x20000000 or ((rows // 128 + chunks + 1) * q_heads > 0xFFFFFF and rows and chunks):
        _refuse_size(f"{what}: more than 2^29 rows, or (rows / 128 + chunks + 1) * q_heads above 2^24 - 1: {rows} rows, "
                     f"{chunks} chunks, {q_heads} heads")
    if sink is not None:
        _check_vector(what, "sink", sink, q_heads, _F32)
    if lse is not None and (lse.dtype != _F32 or lse.shape != (q_heads, rows) or not lse.is_contiguous()):
        _refuse(f"{what}: lse must be contiguous float32 [{q_heads}, {rows}], got {tuple(lse.shape)} {lse.dtype}")
    return rows, q_heads, kv_heads, head_dim


def _pack(what, sizes, q, k, v, cu_seqlens, window, scale, sink, out, lse):
    rows, q_heads, kv_heads, head_dim = sizes
    kv = k.shape
    return _ATTENTION.pack(
        rows, q_heads, kv_heads, head_dim, cu_seqlens.shape[0] - 1,
        -1 if window is None or window < 0 else min(int(window), 0x7FFFFFFF),
        head_dim ** -0.5 if scale is None and head_dim else float(scale or 0.0), cu_seqlens.data_ptr(),
        0 if sink is None else sink.data_ptr(), *_heads(what, "q", q, q.shape), *_heads(what, "k", k, kv),
        *_heads(what, "v", v, kv), *_heads(what, "out", out, q.shape), 0 if lse is None else lse.data_ptr())


def chunk_attention(q, k, v, cu_seqlens, window=-1, scale=None, sink=None, out=None, lse=None,
                    return_lse: bool = False, stream=None):
    """mimo_chunk_attention: attention of every row to the rows of its chunk
    (vision page, MiMoVisionAttention), forward.

    q bf16 [rows, q_heads, head_dim]; k, v bf16 [rows, kv_heads, head_dim],
    each with an innermost axis that is dense and other strides in multiples
    of 8 values (slices of one projection's output are fine); cu_seqlens
    int32 [chunks + 1], ascending within [0, rows] (not checked: the outputs
    are undefined where it is not), on the same GPU (vit_tables' boundaries,
    moved there once).  window >= 0 limits a row to keys at most that far from it in its
    chunk; sink (float32 [q_heads]; beyond +-8192 it counts as that, -inf takes
    key 0 away) is added to each chunk's key 0's logit; scale defaults to
    head_dim ** -0.5.

    Returns out [rows, q_heads, head_dim], or with return_lse=True (out, lse)
    with lse float32 [q_heads, rows], which the backward pass takes.  Rows
    behind cu_seqlens[-1] are left as they were (undefined where out is
    allocated here).
    """
    what = "chunk_attention"
    sizes = _check_qkv(what, q, k, v, cu_seqlens, sink, lse)
    index = q.get_device()
    if (index < 0 or k.get_device() != index or v.get_device() != index or cu_seqlens.get_device() != index
            or (sink is not None and sink.get_device() != index) or (out is not None and out.get_device() != index)
            or (lse is not None and lse.get_device() != index)):
        _heads(what, "q", q, q.shape)
        if out is not None:
            _heads(what, "out", out, q.shape)
        _check_devices(what, (q, k, v, cu_seqlens, sink, out, lse))
    if stream is not None or _device_now() != index:
        with _entered(what, index, stream, (q, k, v, cu_seqlens, sink, out, lse)):
            return chunk_attention(q, k, v, cu_seqlens, window, scale, sink, out, lse, return_lse)
    if out is None:
        out = _dense_like(q)
    if return_lse and lse is None:
        lse = q.new_empty((sizes[1], sizes[0]), dtype=_F32)
    code = _library().mimo_chunk_attention(_pack(what, sizes, q, k, v, cu_seqlens, window, scale, sink, out, lse),
                                           _raw_stream(index))
    if code:
        _abi._check(code, what)
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
    chunk_attention_workspace_bytes(rows, q_heads, kv_heads, head_dim, chunks)
    bytes; calls that may run at the same time need one each.
    """
    what = "chunk_attention_backward"
    if lse is None:
        _refuse(f"{what}: lse is None (chunk_attention returns it with return_lse=True)")
    sizes = _check_qkv(what, q, k, v, cu_seqlens, sink, lse)
    if dsink is not None:
        if sink is None:
            _refuse(f"{what}: dsink is given without sink")
        _check_vector(what, "dsink", dsink, sizes[1], _F32)
    if workspace is not None:
        _abi._check_bytes(workspace, what + ": workspace")
    args = _pack(what, sizes, q, k, v, cu_seqlens, window, scale, sink, out, lse)
    dout_heads = _heads(what, "dout", dout, q.shape)
    index = q.get_device()
    tensors = (q, k, v, out, lse, cu_seqlens, sink, dout, dq, dk, dv, dsink, workspace)
    for t in tensors:
        if t is not None and (index < 0 or t.get_device() != index):
            _check_devices(what, tensors)
    if stream is not None or _device_now() != index:
        with _entered(what, index, stream, tensors):
            return chunk_attention_backward(dout, q, k, v, out, lse, cu_seqlens, window, scale, sink, dq, dk, dv, dsink,
                                            workspace)
    if dq is None:
        dq = _dense_like(q)
    if dk is None:
        dk = _dense_like(k)
    if dv is None:
        dv = _dense_like(v)
    if dsink is None and sink is not None:
        dsink = torch.empty_like(sink)
    lib = _library()
    if workspace is None:
        need = lib.mimo_chunk_attention_workspace_bytes(*sizes, cu_seqlens.shape[0] - 1)
        workspace = q.new_empty(max(need, 16), dtype=torch.uint8)
    grads = _GRADS.pack(*dout_heads, *_heads(what, "dq", dq, q.shape), *_heads(what, "dk", dk, k.shape),
                        *_heads(what, "dv", dv, v.shape), 0 if dsink is None else dsink.data_ptr())
    code = lib.mimo_chunk_attention_backward(args, grads, workspace.data_ptr(), workspace.numel(), _raw_stream(index))
    if code:
        _abi._check(code, what)
    return dq, dk, dv, dsink


def chunk_attention_workspace_bytes(rows: int, q_heads: int, kv_heads: int, head_dim: int, chunks: int) -> int:
    """mimo_chunk_attention_workspace_bytes."""
    return int(_library().mimo_chunk_attention_workspace_bytes(int(rows), int(q_heads), int(kv_heads), int(head_dim), int(chunks)))


# ----------------------------------------------------------------- layer norm

def _out_type(what, out_dtype):
    if out_dtype not in _TYPES:
        _refuse(f"{what}: out_dtype {out_dtype!r} is not f32 or bf16")
    return _TYPES[out_dtype]


def _rows_of(what, x, widest):
    _check_matrix(what, "x", x)
    rows, width = x.shape
    if width < 1:
        _refuse(f"{what}: x has no columns")
    if width > widest or rows > 0x7FFFFFFF:
        _refuse_size(f"{what}: width above {widest} or more than 2^31 - 1 rows: {rows} x {width}")
    return rows, width


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
    rows, width = _rows_of(what, x, 65536)
    if weight is not None:
        _check_vector(what, "weight", weight, width, _F32)
    if bias is not None:
        _check_vector(what, "bias", bias, width, _F32)
    if mean is not None:
        _check_vector(what, "mean", mean, rows, _F32)
    if rstd is not None:
        _check_vector(what, "rstd", rstd, rows, _F32)
    if out is not None:
        _check_matrix(what, "out", out)
        _check_shape(what, "out", out, x.shape)
        dtype = out.dtype
    else:
        dtype = x.dtype if out_dtype is None else _out_type(what, out_dtype)
    index = x.get_device()
    if (index < 0 or (weight is not None and weight.get_device() != index) or (bias is not None and bias.get_device() != index)
            or (out is not None and out.get_device() != index) or (mean is not None and mean.get_device() != index)
            or (rstd is not None and rstd.get_device() != index)):
        _check_devices(what, (x, weight, bias, out, mean, rstd))
    if stream is not None or _device_now() != index:
        with _entered(what, index, stream, (x, weight, bias, out, mean, rstd)):
            return layer_norm(x, weight, bias, eps, out, out_dtype, return_stats, mean, rstd)
    if out is None:
        out = torch.empty_like(x, dtype=dtype)
    if return_stats:
        if mean is None:
            mean = x.new_empty(rows, dtype=_F32)
        if rstd is None:
            rstd = x.new_empty(rows, dtype=_F32)
    code = _library().mimo_layer_norm(rows, width, x.data_ptr(), _CODES[x.dtype], _pointer(weight), _pointer(bias), eps,
                                      _CODES[dtype], out.data_ptr(), _pointer(mean), _pointer(rstd), _raw_stream(index))
    if code:
        _abi._check(code, what)
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
    rows, width = _rows_of(what, x, 65536)
    _check_matrix(what, "dout", dout)
    _check_shape(what, "dout", dout, x.shape)
    if mean is None or rstd is None:
        _refuse(f"{what}: mean and rstd are needed (layer_norm returns them with return_stats=True)")
    _check_vector(what, "mean", mean, rows, _F32)
    _check_vector(what, "rstd", rstd, rows, _F32)
    if weight is not None:
        _check_vector(what, "weight", weight, width, _F32)
    if dweight is not None:
        _check_vector(what, "dweight", dweight, width, _F32)
    if dbias is not None:
        _check_vector(what, "dbias", dbias, width, _F32)
    if dx is not None:
        _check_matrix(what, "dx", dx, (x.dtype,))
        _check_shape(what, "dx", dx, x.shape)
    if workspace is not None:
        _abi._check_bytes(workspace, what + ": workspace")
    index = x.get_device()
    tensors = (x, dout, mean, rstd, weight, dx, dweight, dbias, workspace)
    for t in tensors:
        if t is not None and (index < 0 or t.get_device() != index):
            _check_devices(what, tensors)
    if stream is not None or _device_now() != index:
        with _entered(what, index, stream, tensors):
            return layer_norm_backward(dout, x, mean, rstd, weight, dx, dweight, dbias, affine, workspace)
    if dx is None:
        dx = torch.empty_like(x)
    if weight is not None if affine is None else affine:
        if dweight is None:
            dweight = x.new_empty(width, dtype=_F32)
        if dbias is None:
            dbias = x.new_empty(width, dtype=_F32)
    lib = _library()
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = x.new_empty(max(lib.mimo_layer_norm_workspace_bytes(rows, width), 16), dtype=torch.uint8)
    code = lib.mimo_layer_norm_backward(
        rows, width, x.data_ptr(), _CODES[x.dtype], dout.data_ptr(), _CODES[dout.dtype], _pointer(weight),
        mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _pointer(dweight), _pointer(dbias), _pointer(workspace),
        0 if workspace is None else workspace.numel(), _raw_stream(index))
    if code:
        _abi._check(code, what)
    return dx, dweight, dbias


def layer_norm_workspace_bytes(rows: int, width: int) -> int:
    """mimo_layer_norm_workspace_bytes."""
    return int(_library().mimo_layer_norm_workspace_bytes(int(rows), int(width)))


# ------------------------------------------------------ 8-bit matrix product

def quantize_rows(x, q=None, scale=None, stream=None):
    """mimo_quantize_rows: x [rows, width] (float32 or bf16, contiguous) to
    8-bit integers, row by row: activations, or a weight [out, in] by output
    channels.

    Returns (q, scale): int8 [rows, padded], padded = width rounded up to a
    multiple of 128 (zeros behind width), and float32 [rows]; x is near
    q[:, :width] * scale[:, None].
    """
    what = "quantize_rows"
    rows, width = _rows_of(what, x, 130944)
    padded = (width + 127) & -128
    if q is not None:
        _check_matrix(what, "q", q, (_I8,))
        _check_shape(what, "q", q, (rows, padded))
    if scale is not None:
        _check_vector(what, "scale", scale, rows, _F32)
    index = x.get_device()
    if index < 0 or (q is not None and q.get_device() != index) or (scale is not None and scale.get_device() != index):
        _check_devices(what, (x, q, scale))
    if stream is not None or _device_now() != index:
        with _entered(what, index, stream, (x, q, scale)):
            return quantize_rows(x, q, scale)
    if q is None:
        q = x.new_empty((rows, padded), dtype=_I8)
    if scale is None:
        scale = x.new_empty(rows, dtype=_F32)
    code = _library().mimo_quantize_rows(rows, width, x.data_ptr(), _CODES[x.dtype], q.data_ptr(), scale.data_ptr(),
                                         _raw_stream(index))
    if code:
        _abi._check(code, what)
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
    _check_matrix(what, "xq", xq, (_I8,))
    _check_matrix(what, "wq", wq, (_I8,))
    rows, k = xq.shape
    n, wk = wq.shape
    if wk != k or k < 128 or k % 128 or n < 1:
        _refuse(f"{what}: xq {tuple(xq.shape)} and wq {tuple(wq.shape)} must share a width that is a multiple of 128")
    if k > 130944 or n > 0x1000000 or rows > 0x7FFFFFFF:
        _refuse_size(f"{what}: width above 130944, more than 2^24 channels or 2^31 - 1 rows: xq {tuple(xq.shape)}, wq {tuple(wq.shape)}")
    _check_vector(what, "x_scale", x_scale, rows, _F32)
    _check_vector(what, "w_scale", w_scale, n, _F32)
    if bias is not None:
        _check_vector(what, "bias", bias, n, _F32)
    if out is not None:
        _check_matrix(what, "out", out)
        _check_shape(what, "out", out, (rows, n))
        dtype = out.dtype
    else:
        dtype = _out_type(what, out_dtype)
    index = xq.get_device()
    if (index < 0 or x_scale.get_device() != index or wq.get_device() != index or w_scale.get_device() != index
            or (bias is not None and bias.get_device() != index) or (out is not None and out.get_device() != index)):
        _check_devices(what, (xq, x_scale, wq, w_scale, bias, out))
    if stream is not None or _device_now() != index:
        with _entered(what, index, stream, (xq, x_scale, wq, w_scale, bias, out)):
            return quantized_linear(xq, x_scale, wq, w_scale, bias, out, out_dtype)
    if out is None:
        out = xq.new_empty((rows, n), dtype=dtype)
    code = _library().mimo_quantized_linear(rows, k, xq.data_ptr(), x_scale.data_ptr(), n, wq.data_ptr(), w_scale.data_ptr(),
                                            _pointer(bias), _CODES[dtype], out.data_ptr(), _raw_stream(index))
    if code:
        _abi._check(code, what)
    return out
