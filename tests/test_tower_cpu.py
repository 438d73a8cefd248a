"""What the tower's operators refuse, and with which code: in the C entry
points, before anything touches a GPU, and in the Python functions."""
import ctypes
import struct

import pytest

import vision_image_preprocessing_amd as V

torch = pytest.importorskip("torch")

P = 1 << 20  # an address that is never used: every call here is refused (or has nothing to do) before a launch


def _attention(rows=10, hq=4, hk=2, d=64, chunks=1, window=-1, scale=0.125, cu=P, sink=0, q=None, k=None, v=None, out=None, lse=P):
    dense = lambda i, h: (P + (i << 24), h * d, d)
    return struct.pack("<q5if2Q" + "Qqq" * 4 + "Q", rows, hq, hk, d, chunks, window, scale, cu, sink,
                       *(q or dense(1, hq)), *(k or dense(2, hk)), *(v or dense(3, hk)), *(out or dense(4, hq)), lse)


def _grads(hq=4, hk=2, d=64, dout=None, dq=None, dk=None, dv=None, dsink=0):
    dense = lambda i, h: (P + (i << 24), h * d, d)
    return struct.pack("<" + "Qqq" * 4 + "Q", *(dout or dense(5, hq)), *(dq or dense(6, hq)), *(dk or dense(7, hk)),
                       *(dv or dense(8, hk)), dsink)


def test_structs_are_as_the_header_lays_them_out():
    assert V.tower._ATTENTION.size == 8 + 5 * 4 + 4 + 2 * 8 + 4 * 24 + 8
    assert V.tower._GRADS.size == 4 * 24 + 8


BAD_ATTENTION = [
    (dict(rows=-1), V.MIMO_E_INVALID), (dict(chunks=-1), V.MIMO_E_INVALID), (dict(hq=0), V.MIMO_E_INVALID),
    (dict(hk=0), V.MIMO_E_INVALID), (dict(hq=5), V.MIMO_E_INVALID), (dict(hq=131072, hk=1), V.MIMO_E_INVALID),
    (dict(d=0), V.MIMO_E_INVALID), (dict(d=4), V.MIMO_E_INVALID), (dict(d=68), V.MIMO_E_INVALID),
    (dict(d=136), V.MIMO_E_INVALID), (dict(scale=0.0), V.MIMO_E_INVALID), (dict(scale=-1.0), V.MIMO_E_INVALID),
    (dict(scale=float("nan")), V.MIMO_E_INVALID), (dict(scale=float("inf")), V.MIMO_E_INVALID),
    (dict(cu=0), V.MIMO_E_INVALID), (dict(cu=P + 2), V.MIMO_E_INVALID), (dict(sink=P + 1), V.MIMO_E_INVALID),
    (dict(rows=(1 << 29) + 1), V.MIMO_E_TOO_LARGE), (dict(rows=1 << 29, hq=65536, hk=1), V.MIMO_E_TOO_LARGE),
    (dict(chunks=(1 << 29) + 1), V.MIMO_E_TOO_LARGE), (dict(rows=1 << 20, chunks=1 << 22, hq=4), V.MIMO_E_TOO_LARGE),
    (dict(q=(0, 256, 64)), V.MIMO_E_INVALID), (dict(q=(P + 8, 256, 64)), V.MIMO_E_INVALID),
    (dict(k=(P, 132, 64)), V.MIMO_E_INVALID), (dict(k=(P, 128, 60)), V.MIMO_E_INVALID),
    (dict(v=(P, 56, 64)), V.MIMO_E_INVALID), (dict(v=(P, 0, 64)), V.MIMO_E_INVALID),
    (dict(v=(P, 128, -64)), V.MIMO_E_INVALID), (dict(q=(P, (1 << 22) + 8, 64)), V.MIMO_E_INVALID),
    (dict(out=(P, 64, 64)), V.MIMO_E_INVALID), (dict(out=(P, 256, 0)), V.MIMO_E_INVALID),
    (dict(out=(P, 128, 64)), V.MIMO_E_INVALID), (dict(out=(0, 256, 64)), V.MIMO_E_INVALID),
    (dict(out=(P + (1 << 24), 256, 64)), V.MIMO_E_INVALID), (dict(lse=P + 2), V.MIMO_E_INVALID),
]


@pytest.mark.parametrize("bad,code", BAD_ATTENTION)
def test_attention_refuses(bad, code):
    lib = V.load()
    before = V.dispatch_count()
    assert lib.mimo_chunk_attention(_attention(**bad), None) == code
    assert V.last_error().startswith("chunk_attention:") and V.dispatch_count() == before


@pytest.mark.parametrize("bad,code", [b for b in BAD_ATTENTION if "out" not in b[0] and "lse" not in b[0]])
def test_attention_backward_refuses_the_same(bad, code):
    assert V.load().mimo_chunk_attention_backward(_attention(**bad), _grads(), P, 1 << 40, None) == code


@pytest.mark.parametrize("bad", [
    dict(dout=(0, 256, 64)), dict(dq=(P + 4, 256, 64)), dict(dk=(P, 128, 0)), dict(dv=(P, 64, 64)), dict(dsink=P + 2),
    dict(dsink=P), dict(dq=(P + (1 << 24), 256, 64)), dict(dk=(P + (8 << 24), 128, 64)), dict(dv=(P + (5 << 24), 128, 64)),
])
def test_attention_backward_refuses(bad):
    # a dsink without a sink among them
    assert V.load().mimo_chunk_attention_backward(_attention(), _grads(**bad), P, 1 << 40, None) == V.MIMO_E_INVALID


def test_attention_backward_refuses_the_sink_as_its_gradient():
    # workgroups that read the sink run next to the ones that write dsink
    assert V.load().mimo_chunk_attention_backward(_attention(sink=P), _grads(dsink=P), P, 1 << 40, None) == V.MIMO_E_INVALID


def test_attention_backward_workspace_and_nulls():
    lib = V.load()
    need = V.chunk_attention_workspace_bytes(10, 4, 2, 64, 1)
    assert need >= 10 * 4 * 4
    assert lib.mimo_chunk_attention_backward(_attention(), _grads(), P, need - 1, None) == V.MIMO_E_CAPACITY
    assert lib.mimo_chunk_attention_backward(_attention(), _grads(), None, need, None) == V.MIMO_E_INVALID
    assert lib.mimo_chunk_attention_backward(_attention(), _grads(), P + 8, need, None) == V.MIMO_E_INVALID
    assert lib.mimo_chunk_attention_backward(_attention(lse=0), _grads(), P, need, None) == V.MIMO_E_INVALID
    assert lib.mimo_chunk_attention_backward(_attention(), None, P, need, None) == V.MIMO_E_INVALID
    assert lib.mimo_chunk_attention_backward(None, _grads(), P, need, None) == V.MIMO_E_INVALID
    assert lib.mimo_chunk_attention(None, None) == V.MIMO_E_INVALID
    for bad in ((-1, 4, 2, 64, 1), (1, 0, 1, 64, 1), (1, 4, 3, 64, 1), (1, 1, 1, 60, 1), (1, 1, 1, 136, 1), (1, 1, 1, 64, -1),
                ((1 << 30) + 1, 1, 1, 64, 1)):
        assert V.chunk_attention_workspace_bytes(*bad) == 0
    # nothing to do: no pointer is looked at
    assert lib.mimo_chunk_attention(_attention(rows=0, cu=0, q=(0, 8, 0)), None) == V.MIMO_OK
    assert lib.mimo_chunk_attention(_attention(chunks=0, cu=0), None) == V.MIMO_OK
    assert lib.mimo_chunk_attention_backward(_attention(rows=0), _grads(), None, 0, None) == V.MIMO_OK


def test_workspace_bytes_are_zero_from_the_first_refused_size_on():
    lib = V.load()
    sizes = lambda rows, chunks, hq, hk=1: (rows, hq, hk, 64, chunks)
    refused = lambda rows, chunks, hq, hk=1: lib.mimo_chunk_attention_backward(
        _attention(rows=rows, chunks=chunks, hq=hq, hk=hk), _grads(hq=hq, hk=hk), P, 0, None)
    for last, first in (((32511, 1, 65536), (32512, 1, 65536)), ((10, (1 << 22) - 2, 4), (10, (1 << 22) - 1, 4)),
                        (((1 << 29), 1, 1), ((1 << 29) + 1, 1, 1)), ((1 << 28, 8, 7), (1 << 29, 8, 7))):
        assert V.chunk_attention_workspace_bytes(*sizes(*last)) > 0 and refused(*last) == V.MIMO_E_CAPACITY
        assert V.chunk_attention_workspace_bytes(*sizes(*first)) == 0 and refused(*first) == V.MIMO_E_TOO_LARGE
    # nothing to do, and so nothing to hold
    assert V.chunk_attention_workspace_bytes(*sizes(0, 1 << 29, 65536)) == 0 and refused(0, 1 << 29, 65536) == V.MIMO_OK
    assert V.chunk_attention_workspace_bytes(*sizes(1 << 29, 0, 65536)) == 0 and refused(1 << 29, 0, 65536) == V.MIMO_OK

    def norm(rows, width):
        return lib.mimo_layer_norm_backward(rows, width, P, V.MIMO_F32, 2 * P, V.MIMO_F32, P, P, P, 3 * P, P, 4 * P, P, 0, None)

    for last, first in ((((1 << 31) - 1, 8), (1 << 31, 8)), ((5, 65536), (5, 65537))):
        assert V.layer_norm_workspace_bytes(*last) > 0 and norm(*last) == V.MIMO_E_CAPACITY
        assert V.layer_norm_workspace_bytes(*first) == 0 and norm(*first) == V.MIMO_E_TOO_LARGE


def test_norm_refuses():
    lib = V.load()
    F, B = V.MIMO_F32, V.MIMO_BF16

    def forward(rows=4, width=64, x=P, xd=F, w=P, b=P, eps=1e-6, od=F, out=2 * P, mean=P, rstd=4 * P):
        return lib.mimo_layer_norm(rows, width, x, xd, w, b, eps, od, out, mean, rstd, None)

    for bad in (dict(rows=-1), dict(width=0), dict(xd=2), dict(od=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(out=None), dict(x=P + 2), dict(xd=B, x=P + 1), dict(out=P + 2),
                dict(w=P + 1), dict(b=P + 2), dict(mean=P + 1), dict(rstd=P + 2), dict(out=P, od=B), dict(rstd=P)):
        assert forward(**bad) == V.MIMO_E_INVALID, bad
    assert forward(width=65537) == V.MIMO_E_TOO_LARGE and forward(rows=1 << 31) == V.MIMO_E_TOO_LARGE
    assert forward(rows=0, x=None, out=None) == V.MIMO_OK

    need = V.layer_norm_workspace_bytes(4, 64)
    assert need >= 2 * 64 * 4 and V.layer_norm_workspace_bytes(-1, 64) == 0 and V.layer_norm_workspace_bytes(4, 65537) == 0

    def backward(rows=4, width=64, x=P, xd=F, g=2 * P, gd=F, w=P, mean=P, rstd=P, dx=3 * P, dw=P, db=4 * P, ws=P, n=need):
        return lib.mimo_layer_norm_backward(rows, width, x, xd, g, gd, w, mean, rstd, dx, dw, db, ws, n, None)

    for bad in (dict(rows=-1), dict(width=0), dict(xd=7), dict(gd=2), dict(x=None), dict(g=None), dict(mean=None),
                dict(rstd=None), dict(dx=None), dict(dx=P), dict(dx=2 * P), dict(dw=P + 2), dict(db=P + 1), dict(ws=None),
                dict(ws=P + 8), dict(x=P + 2), dict(gd=B, g=P + 1), dict(w=P + 2), dict(mean=P + 2),
                dict(db=P)):
        assert backward(**bad) == V.MIMO_E_INVALID, bad
    assert backward(n=need - 1) == V.MIMO_E_CAPACITY
    assert backward(width=65537) == V.MIMO_E_TOO_LARGE
    assert backward(rows=0, dw=None, db=None) == V.MIMO_OK


def test_quantized_refuses():
    lib = V.load()

    def quantize(rows=4, width=64, x=P, d=V.MIMO_F32, q=2 * P, s=P):
        return lib.mimo_quantize_rows(rows, width, x, d, q, s, None)

    for bad in (dict(rows=-1), dict(width=0), dict(d=2), dict(x=None), dict(q=None), dict(s=None), dict(x=P + 2),
                dict(x=P + 1, d=V.MIMO_BF16), dict(q=P + 8), dict(s=P + 2), dict(q=P)):
        assert quantize(**bad) == V.MIMO_E_INVALID, bad
    assert quantize(width=130945) == V.MIMO_E_TOO_LARGE and quantize(rows=1 << 31) == V.MIMO_E_TOO_LARGE
    assert quantize(rows=0, x=None) == V.MIMO_OK

    def linear(rows=4, k=128, x=P, xs=P, e=8, w=2 * P, ws=P, b=P, d=V.MIMO_F32, out=3 * P):
        return lib.mimo_quantized_linear(rows, k, x, xs, e, w, ws, b, d, out, None)

    for bad in (dict(rows=-1), dict(k=0), dict(k=64), dict(k=130), dict(e=0), dict(d=2), dict(x=None), dict(xs=None),
                dict(w=None), dict(ws=None), dict(out=None), dict(x=P + 8), dict(w=P + 8), dict(out=P + 8), dict(b=P + 2),
                dict(xs=P + 2), dict(ws=P + 1), dict(out=P), dict(out=2 * P)):
        assert linear(**bad) == V.MIMO_E_INVALID, bad
    assert linear(k=131072) == V.MIMO_E_TOO_LARGE and linear(e=(1 << 24) + 1) == V.MIMO_E_TOO_LARGE
    assert linear(rows=0, x=None, out=None) == V.MIMO_OK


def _refused(f, *a, **k):
    with pytest.raises(V.MimoError) as e:
        f(*a, **k)
    assert e.value.code == V.MIMO_E_INVALID
    return str(e.value)


def test_python_checks():
    """Shapes and types first, then devices: host tensors that are otherwise
    fine are refused as such."""
    bf = torch.bfloat16
    q, k = torch.zeros((6, 4, 64), dtype=bf), torch.zeros((6, 2, 64), dtype=bf)
    cu = torch.tensor([0, 6], dtype=torch.int32)
    att = lambda q=q, k=k, v=k, cu=cu, **kw: _refused(V.chunk_attention, q, k, v, cu, **kw)
    assert "one GPU" in att()
    assert "q must be" in att(q=q.float())
    assert "k must be" in att(k=k[:, :, 0])
    assert "agree" in att(k=k[:5]) and "agree" in att(k=torch.zeros((6, 3, 64), dtype=bf))
    assert "v must be" in att(v=torch.zeros((6, 2, 32), dtype=bf))
    assert "dense" in att(q=q.transpose(1, 2).contiguous().transpose(1, 2))
    assert "cu_seqlens" in att(cu=cu.long()) and "cu_seqlens" in att(cu=cu[:0]) and "cu_seqlens" in att(cu=torch.zeros(6, dtype=torch.int32)[::2])
    assert "sink" in att(sink=torch.zeros(3)) and "sink" in att(sink=torch.zeros(4, dtype=bf))
    assert "lse" in att(lse=torch.zeros(6, 4)) and "out must be" in att(out=q[:5])
    lse = torch.zeros(4, 6)
    back = lambda dout=q, out=q, lse=lse, **kw: _refused(V.chunk_attention_backward, dout, q, k, k, out, lse, cu, **kw)
    assert "one GPU" in back()
    assert "dout must be" in back(dout=q[:, :2]) and "lse" in back(lse=None) and "dsink" in back(dsink=torch.zeros(4))
    x = torch.zeros(4, 64)
    norm = lambda x=x, *a, **kw: _refused(V.layer_norm, x, *a, **kw)
    assert "one GPU" in norm()
    assert "x must be" in norm(x[0]) and "x must be" in norm(x.double()) and "x must be" in norm(x.t())
    assert "no columns" in norm(x[:, :0].contiguous())
    assert "weight" in norm(x, torch.zeros(63)) and "bias" in norm(x, None, torch.zeros(64, dtype=bf))
    assert "out_dtype" in norm(out_dtype="f16") and "out must be" in norm(out=x[:3])
    m = torch.zeros(4)
    nback = lambda dout=x, x=x, mean=m, rstd=m, **kw: _refused(V.layer_norm_backward, dout, x, mean, rstd, **kw)
    assert "one GPU" in nback()
    assert "dout must be" in nback(dout=x[:3]) and "mean" in nback(mean=m[:3]) and "needed" in nback(rstd=None)
    assert "dx must be" in nback(dx=x.to(bf)) and "dweight" in nback(dweight=m)
    assert "one GPU" in _refused(V.quantize_rows, x) and "x must be" in _refused(V.quantize_rows, x.half())
    assert "q must be" in _refused(V.quantize_rows, x, q=torch.zeros((4, 64), dtype=torch.int8))
    i = torch.zeros((4, 128), dtype=torch.int8)
    lin = lambda a=i, s=m, w=i, t=m, **kw: _refused(V.quantized_linear, a, s, w, t, **kw)
    assert "one GPU" in lin()
    assert "multiple of 128" in lin(i[:, :64].contiguous(), m, i[:, :64].contiguous()) and "xq must be" in lin(i.float())
    assert "x_scale" in lin(s=m[:3]) and "w_scale" in lin(t=m.double()) and "bias" in lin(bias=m[:2])
    assert "out_dtype" in lin(out_dtype="i8") and "out must be" in lin(out=torch.zeros(4, 5))


def test_python_refuses_sizes_before_it_allocates():
    """Outputs, gradients and workspaces of these would be terabytes."""
    bf, meta = torch.bfloat16, dict(device="meta")

    def too_large(f, *a, **k):
        with pytest.raises(V.MimoError) as e:
            f(*a, **k)
        assert e.value.code == V.MIMO_E_TOO_LARGE and str(e.value)

    def attention(rows, chunks, hq):
        q = torch.zeros((rows, 1, 128), dtype=bf, **meta).expand(rows, hq, 128)
        k, cu = torch.zeros((rows, 1, 128), dtype=bf, **meta), torch.zeros(chunks + 1, dtype=torch.int32, **meta)
        return q, k, cu, torch.zeros((hq, rows), **meta)

    for size in ((32512, 1, 65536), (1 << 28, 8, 8), ((1 << 29) + 1, 1, 1), (10, (1 << 22) - 1, 4)):
        q, k, cu, lse = attention(*size)
        too_large(V.chunk_attention, q, k, k, cu)
        too_large(V.chunk_attention_backward, q, q, k, k, q, lse, cu)
    # the last size below, and nothing to do, are refused for their device alone
    for size in ((32511, 1, 65536), (0, 1 << 22, 65536), (1 << 29, 0, 8)):
        q, k, cu, lse = attention(*size)
        assert "one GPU" in _refused(V.chunk_attention, q, k, k, cu)
        assert "one GPU" in _refused(V.chunk_attention_backward, q, q, k, k, q, lse, cu)
    for rows, width, quantized in ((1 << 31, 1, True), (2, 65537, False), (2, 130945, True)):
        x, m = torch.zeros((rows, width), **meta), torch.zeros(rows, **meta)
        if not quantized or width == 1:
            too_large(V.layer_norm, x)
            too_large(V.layer_norm_backward, x, x, m, m)
        if quantized:
            too_large(V.quantize_rows, x)
    x = torch.zeros((2, 130944), **meta)
    assert "one GPU" in _refused(V.quantize_rows, x) and "one GPU" in _refused(V.layer_norm, x[:, :65536].contiguous())
    i, m = torch.zeros((4, 131072), dtype=torch.int8, **meta), torch.zeros(4, **meta)
    too_large(V.quantized_linear, i, m, i, m)
    i, n = torch.zeros((4, 128), dtype=torch.int8, **meta), (1 << 24) + 1
    too_large(V.quantized_linear, i, m, torch.zeros((n, 128), dtype=torch.int8, **meta), torch.zeros(n, **meta))


def test_names_are_exported():
    for name in V._TOWER:
        assert callable(getattr(V, name)) and name in dir(V)
    with pytest.raises(AttributeError):
        V.no_such_operator
