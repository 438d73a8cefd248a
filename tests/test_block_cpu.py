"""What the block's operators refuse, and with which code: in the C entry
points, before anything touches a GPU, and in the Python functions."""
import struct

import pytest

import vision_image_preprocessing_amd as V

torch = pytest.importorskip("torch")

P = 1 << 20  # an address that is never used: every call here is refused (or has nothing to do) before a launch
F, B = V.MIMO_F32, V.MIMO_BF16


def _forward(rows=4, width=64, x=P, xd=F, r=2 * P, rd=F, w=3 * P, eps=1e-6, h=4 * P, od=F, out=5 * P, rstd=6 * P):
    return V.load().mimo_rms_norm(rows, width, x, xd, r, rd, w, eps, h, od, out, rstd, None)


def _quantized(rows=4, width=64, x=P, xd=F, r=2 * P, rd=F, w=3 * P, eps=1e-6, h=4 * P, q=5 * P, s=6 * P):
    return V.load().mimo_rms_norm_quantized(rows, width, x, xd, r, rd, w, eps, h, q, s, None)


BOTH = [dict(rows=-1), dict(width=0), dict(xd=2), dict(xd=-1), dict(rd=3), dict(rd=B), dict(eps=-1.0), dict(eps=float("nan")),
        dict(eps=float("inf")), dict(x=None), dict(x=P + 2), dict(xd=B, x=P + 1), dict(r=2 * P + 2), dict(xd=B, rd=B, r=P + 1),
        dict(h=None), dict(h=4 * P + 1), dict(w=P + 2), dict(xd=B, h=P), dict(h=5 * P)]


@pytest.mark.parametrize("bad", BOTH + [dict(od=2), dict(od=-1), dict(out=None), dict(out=P + 2), dict(rstd=P + 1),
                                        dict(out=P, od=B), dict(out=2 * P, od=B), dict(out=3 * P), dict(rstd=3 * P), dict(h=3 * P)])
def test_norm_refuses(bad):
    before = V.dispatch_count()
    assert _forward(**bad) == V.MIMO_E_INVALID
    assert V.last_error().startswith("rms_norm:") and V.dispatch_count() == before


@pytest.mark.parametrize("bad", BOTH + [dict(q=None), dict(q=P + 8), dict(q=P), dict(q=2 * P), dict(s=None), dict(s=P + 2), dict(q=3 * P), dict(s=3 * P),
                                        dict(h=3 * P)])
def test_quantized_norm_refuses(bad):
    assert _quantized(**bad) == V.MIMO_E_INVALID and V.last_error().startswith("rms_norm_quantized:")


def test_norm_refuses_outputs_that_are_one_array():
    """What is written a value a row is no array whose other rows are read."""
    for at in (P, 2 * P, 4 * P, 5 * P):
        assert _forward(rstd=at) == V.MIMO_E_INVALID and V.last_error().startswith("rms_norm: rstd")
        assert _quantized(s=at) == V.MIMO_E_INVALID and V.last_error().startswith("rms_norm_quantized: scale")
    need = V.rms_norm_workspace_bytes(4, 64)
    for dweight in (P, 2 * P, 5 * P, 6 * P):
        assert V.load().mimo_rms_norm_backward(4, 64, P, F, 2 * P, F, 3 * P, 4 * P, 5 * P, 6 * P, dweight, 8 * P, need,
                                               None) == V.MIMO_E_INVALID
        assert V.last_error().startswith("rms_norm_backward: dweight")


def test_norm_sizes():
    for call in (_forward, _quantized):
        assert call(width=65537) == V.MIMO_E_TOO_LARGE and call(rows=1 << 31) == V.MIMO_E_TOO_LARGE
        assert call(rows=0, x=None, r=None, h=None) == V.MIMO_OK


def test_norm_backward_refuses():
    lib = V.load()
    need = V.rms_norm_workspace_bytes(4, 64)
    assert need >= 64 * 4 and V.rms_norm_workspace_bytes(-1, 64) == 0
    assert V.rms_norm_workspace_bytes(4, 65537) == 0 and V.rms_norm_workspace_bytes(1 << 31, 4) == 0

    def backward(rows=4, width=64, h=P, hd=F, g=2 * P, gd=F, w=3 * P, rstd=4 * P, dr=5 * P, dx=6 * P, dw=7 * P, ws=P, n=need):
        return lib.mimo_rms_norm_backward(rows, width, h, hd, g, gd, w, rstd, dr, dx, dw, ws, n, None)

    for bad in (dict(rows=-1), dict(width=0), dict(hd=7), dict(gd=2), dict(h=None), dict(g=None), dict(rstd=None), dict(dx=None),
                dict(dx=P), dict(dx=2 * P), dict(dw=P + 2), dict(ws=None), dict(ws=P + 8), dict(h=P + 2), dict(gd=B, g=P + 1),
                dict(w=P + 2), dict(rstd=P + 2), dict(dr=P + 2), dict(dw=3 * P), dict(dw=4 * P), dict(dx=3 * P), dict(dx=4 * P)):
        assert backward(**bad) == V.MIMO_E_INVALID, bad
    assert backward(n=need - 1) == V.MIMO_E_CAPACITY
    assert backward(width=65537) == V.MIMO_E_TOO_LARGE and backward(rows=1 << 31) == V.MIMO_E_TOO_LARGE
    assert backward(rows=0, dw=None, h=None, dx=None) == V.MIMO_OK


def test_rotation_refuses():
    lib = V.load()
    heads = lambda p=P, row=256, head=64: struct.pack("<Qqq", p, row, head)

    def rotate(rows=10, n=4, d=64, x=heads(), cos=2 * P, sin=3 * P, out=heads(4 * P)):
        return lib.mimo_rotate_heads(rows, n, d, x, cos, sin, 0, out, None)

    before = V.dispatch_count()
    for bad in (dict(rows=-1), dict(n=0), dict(n=65537), dict(d=0), dict(d=4), dict(d=60), dict(d=520), dict(x=None), dict(out=None),
                dict(x=heads(0)), dict(x=heads(P + 8)), dict(x=heads(P, 252)), dict(x=heads(P, 56)), dict(x=heads(P, 256, 60)),
                dict(x=heads(P, 256, -64)), dict(x=heads(P, (1 << 22) + 8)), dict(out=heads(0)), dict(out=heads(4 * P, 64)),
                dict(out=heads(4 * P, 256, 0)), dict(out=heads(4 * P, 192)), dict(out=heads(P, 512)), dict(out=heads(P, 264, 64)),
                dict(out=heads(4 * P, 64, 576)), dict(cos=None), dict(sin=None), dict(cos=P + 4), dict(sin=P + 8)):
        assert rotate(**bad) == V.MIMO_E_INVALID, bad
        assert V.last_error().startswith("rotate_heads:")
    assert rotate(rows=(1 << 29) + 1) == V.MIMO_E_TOO_LARGE
    assert rotate(rows=0, x=heads(0), cos=None) == V.MIMO_OK and V.dispatch_count() == before


def test_functions_refuse_what_is_not_on_a_gpu():
    x, w = torch.zeros((4, 64)), torch.ones(64)
    for call in (lambda: V.rms_norm(x, w), lambda: V.rms_norm(x, w, x), lambda: V.rms_norm_quantized(x, w),
                 lambda: V.rms_norm_backward(x, x, torch.ones(4), w),
                 lambda: V.rotate_heads(torch.zeros((4, 2, 32), dtype=torch.bfloat16), torch.zeros((4, 16)), torch.zeros((4, 16)))):
        with pytest.raises(Exception):
            call()


def _mlp(rows=4, width=64, hidden=72, x=P, wg=2 * P, wu=3 * P, wd=4 * P, bg=5 * P, bu=6 * P, bd=7 * P, gu=8 * P, h=9 * P):
    return V.tower._MLP.pack(rows, width, hidden, x, wg, wu, wd, bg, bu, bd, gu, h)


def _mlp_grads(dout=11 * P, dx=12 * P, dwg=13 * P, dwu=14 * P, dwd=15 * P, dbg=16 * P, dbu=17 * P, dbd=18 * P):
    return V.tower._MLP_GRADS.pack(dout, dx, dwg, dwu, dwd, dbg, dbu, dbd)


def test_mlp_refuses():
    lib = V.load()
    need = V.gated_mlp_workspace_bytes(4, 64, 72)
    assert need >= 4 * 128 * 2

    def forward(out=10 * P, ws=20 * P, n=need, **kw):
        return lib.mimo_gated_mlp(_mlp(**kw), out, ws, n, None)

    before = V.dispatch_count()
    for bad in (dict(rows=-1), dict(width=0), dict(hidden=0), dict(x=0), dict(wg=0), dict(wu=0), dict(wd=0), dict(out=None), dict(x=P + 8),
                dict(wg=P + 2), dict(wu=P + 4), dict(wd=P + 8), dict(out=P + 8), dict(bg=P + 2), dict(bu=P + 1), dict(bd=P + 2), dict(gu=0),
                dict(h=0), dict(gu=P + 8), dict(h=P + 8), dict(out=P), dict(out=2 * P), dict(out=3 * P), dict(out=4 * P), dict(out=8 * P),
                dict(out=9 * P), dict(ws=None), dict(ws=P + 8), dict(h=P), dict(h=8 * P), dict(gu=4 * P), dict(out=7 * P), dict(h=5 * P)):
        assert forward(**bad) == V.MIMO_E_INVALID, bad
        assert V.last_error().startswith("gated_mlp:")
    assert forward(n=need - 1) == V.MIMO_E_CAPACITY and lib.mimo_gated_mlp(None, P, P, need, None) == V.MIMO_E_INVALID
    for bad in (dict(rows=1 << 31), dict(width=65537), dict(hidden=65537), dict(rows=1 << 30, hidden=65536)):
        assert forward(**bad) == V.MIMO_E_TOO_LARGE, bad
    assert forward(rows=0, x=0, out=None, ws=None) == V.MIMO_OK and V.dispatch_count() == before
    for sizes in ((-1, 64, 72), (4, 0, 72), (4, 64, 0), (1 << 31, 64, 72), (4, 65537, 72), (4, 64, 65537), (1 << 30, 64, 65536)):
        assert V.gated_mlp_workspace_bytes(*sizes) == 0 and V.gated_mlp_backward_workspace_bytes(*sizes) == 0


def test_mlp_tiles():
    """A workgroup of a 256 x 256 tile has 512 threads, and a launch fewer than
    2^32: one more row of tiles than fits is refused."""
    rows = 256 * ((1 << 23) // (1 + 1))  # tiles of 128 hidden values and of 256 outputs
    assert V.gated_mlp_workspace_bytes(rows, 256, 128) == 0 and V.gated_mlp_backward_workspace_bytes(rows, 256, 128) == 0
    assert V.gated_mlp_workspace_bytes(rows - 256, 256, 128) > 0 and V.gated_mlp_backward_workspace_bytes(rows - 256, 256, 128) > 0
    assert V.load().mimo_gated_mlp(_mlp(rows=rows, width=256, hidden=128), 10 * P, 20 * P, 1 << 62, None) == V.MIMO_E_TOO_LARGE
    # in Python before outputs of such a size are allocated
    x, w, wd = (torch.empty(s, dtype=torch.bfloat16, device="meta") for s in ((rows, 256), (128, 256), (256, 128)))
    gate_up, hidden = torch.empty((2, rows, 128), device="meta"), torch.empty((rows, 128), dtype=torch.bfloat16, device="meta")
    for call in (lambda: V.gated_mlp(x, w, w, wd), lambda: V.gated_mlp_backward(x, x, w, w, wd, gate_up, hidden)):
        with pytest.raises(V.MimoError) as error:
            call()
        assert error.value.code == V.MIMO_E_TOO_LARGE


def test_mlp_backward_refuses():
    lib = V.load()
    need = V.gated_mlp_backward_workspace_bytes(4, 64, 72)
    assert need >= 2 * 4 * 128 * 2

    def backward(args=None, ws=20 * P, n=need, **kw):
        return lib.mimo_gated_mlp_backward(_mlp(**(args or {})), _mlp_grads(**kw), ws, n, None)

    for bad in (dict(rows=-1), dict(width=0), dict(x=0), dict(wg=0), dict(wu=0), dict(wd=0), dict(gu=0), dict(h=0), dict(x=P + 8), dict(h=P + 8)):
        assert backward(args=bad) == V.MIMO_E_INVALID, bad
        assert V.last_error().startswith("gated_mlp_backward:")
    for bad in (dict(dout=0), dict(dout=P + 8), dict(dx=P + 8), dict(dwg=P + 2), dict(dwu=P + 4), dict(dwd=P + 8), dict(dbg=P + 2), dict(dbu=P + 1),
                dict(dbd=P + 2), dict(dx=P), dict(dx=11 * P), dict(dwg=2 * P), dict(dwd=9 * P), dict(dx=8 * P), dict(dwg=14 * P), dict(dbg=17 * P),
                dict(dx=15 * P), dict(ws=None), dict(ws=P + 8)):
        assert backward(**bad) == V.MIMO_E_INVALID, bad
    assert backward(n=need - 1) == V.MIMO_E_CAPACITY
    assert lib.mimo_gated_mlp_backward(_mlp(), None, P, need, None) == V.MIMO_E_INVALID
    assert lib.mimo_gated_mlp_backward(None, _mlp_grads(), P, need, None) == V.MIMO_E_INVALID
    assert backward(args=dict(width=65537)) == V.MIMO_E_TOO_LARGE
    assert backward(args=dict(rows=0), dwg=0, dwu=0, dwd=0, dbg=0, dbu=0, dbd=0, ws=None) == V.MIMO_OK


def test_mlp_structs_are_as_the_header_lays_them_out():
    assert V.tower._MLP.size == 16 + 9 * 8 and V.tower._MLP_GRADS.size == 8 * 8


def _overlap_refused(rows, n, d, x, out):
    """Whether the rotation refuses (base, row stride, head stride), in values,
    for where they lie: looked at before the tables, which are missing here, so
    that no call gets further."""
    pack = lambda t: struct.pack("<Qqq", P + 2 * t[0], t[1], t[2])
    assert V.load().mimo_rotate_heads(rows, n, d, pack(x), None, None, 0, pack(out), None) == V.MIMO_E_INVALID
    message = V.last_error()
    assert "overlap" in message or "cos and sin" in message, message
    return "overlap" in message


def test_rotation_refuses_out_that_overlaps_x_in_part():
    """Eight heads further in the same rows is written over what others read;
    the heads behind x's, in x's rows, are not."""
    row = 48 * 64
    for shift, refused in ((8, True), (16, True), (40, False), (-8, True)):
        assert _overlap_refused(1001, 40 if shift != 40 else 8, 64, (1 << 20, row, 64), ((1 << 20) + shift * 64, row, 64)) == refused
    assert not _overlap_refused(1001, 8, 64, (40 * 64, row, 64), (0, row, 64))
    # the next rows of one array; a head's halves
    assert _overlap_refused(100, 4, 64, (0, 256, 64), (256, 256, 64)) and not _overlap_refused(100, 4, 64, (0, 256, 64), (25600, 256, 64))
    assert _overlap_refused(1, 1, 64, (0, 64, 64), (8, 64, 64)) and not _overlap_refused(1, 1, 64, (0, 64, 64), (64, 64, 64))
    # one head, read again and again, and the heads behind it; every second head
    assert not _overlap_refused(100, 4, 64, (0, 320, 0), (64, 320, 64)) and _overlap_refused(100, 4, 64, (64, 320, 0), (64 * 2 - 8, 320, 64))
    assert not _overlap_refused(100, 4, 64, (0, 1024, 128), (64, 1024, 128)) and not _overlap_refused(9, 4, 64, (0, 1024, 128), (512, 1024, 64))


def test_rotation_tells_what_overlaps():
    """Small tensors at every kind of place in one array, against the sets of
    their values: none that overlaps passes, and of those with one row stride
    whose heads lie within it, or that have one head stride too, none that does
    not is refused."""
    import random

    rng = random.Random(5)
    told = 0
    for _ in range(6000):
        rows, n, d = rng.randint(1, 4), rng.randint(1, 4), rng.choice([8, 16])
        strides = []
        for _ in range(2):
            head = 8 * rng.randint(d // 8, 6)
            turned = rng.random() < 0.3
            row = 8 * rng.randint(d // 8, 30)
            if turned:
                head = (rows - 1) * row + d + 8 * rng.randint(0, 12)
            else:
                row = max(row, (n - 1) * head + d)
            strides.append((row, head))
        if rng.random() < 0.7:
            strides[0] = strides[1] if rng.random() < 0.5 else (strides[1][0], strides[0][1])
        if rng.random() < 0.2:
            strides[0] = (strides[0][0], 0)
        x, out = (512, *strides[0]), (512 + 8 * rng.randint(-60, 60), *strides[1])
        if x[0] == out[0]:
            continue
        values = [{t[0] + r * t[1] + h * t[2] + i for r in range(rows) for h in range(n) for i in range(d)} for t in (x, out)]
        meet = bool(values[0] & values[1])
        refused = _overlap_refused(rows, n, d, x, out)
        assert refused or not meet, (rows, n, d, x, out)
        inside = all((n - 1) * t[2] + d <= t[1] for t in (x, out))
        if rows == 1 or (x[1] == out[1] and (inside or n == 1 or x[2] == out[2])):
            assert refused == meet, (rows, n, d, x, out)
            told += not meet
    assert told > 300


def test_rotation_refuses_tables_among_the_outputs():
    heads = lambda p: struct.pack("<Qqq", p, 256, 64)
    for cos, sin in ((4 * P, 3 * P), (2 * P, 4 * P + 16), (4 * P - 1264, 3 * P)):
        assert V.load().mimo_rotate_heads(10, 4, 64, heads(P), cos, sin, 0, heads(4 * P), None) == V.MIMO_E_INVALID
        assert V.last_error().startswith("rotate_heads: cos and sin must not lie")


def test_norm_refuses_arrays_that_overlap_in_part():
    """4 rows of 64 float32 values are 1024 bytes, the weight 256, rstd and
    scale 16, 8-bit rows 512: one more or one less address further."""
    for bad in (dict(out=P + 4), dict(out=P - 1020), dict(out=2 * P + 1020), dict(out=3 * P - 1020), dict(out=3 * P + 252), dict(out=4 * P + 1020),
                dict(out=6 * P - 1020), dict(h=P + 4), dict(h=2 * P + 512), dict(h=3 * P + 252), dict(rstd=P + 1020), dict(rstd=2 * P - 12),
                dict(rstd=3 * P + 252), dict(rstd=4 * P + 4), dict(rstd=5 * P - 12), dict(xd=B, rd=B, od=B, out=P + 510)):
        assert _forward(**bad) == V.MIMO_E_INVALID and V.last_error().startswith("rms_norm:"), bad
        assert "in part" in V.last_error()
    for bad in (dict(q=P + 16), dict(q=2 * P - 496), dict(q=3 * P + 240), dict(q=4 * P + 1008), dict(h=P + 4), dict(h=3 * P - 4), dict(s=P + 1020),
                dict(s=2 * P + 4), dict(s=3 * P + 252), dict(s=4 * P - 12), dict(s=5 * P + 508), dict(xd=B, rd=B, q=2 * P + 496)):
        assert _quantized(**bad) == V.MIMO_E_INVALID and V.last_error().startswith("rms_norm_quantized:"), bad
        assert "in part" in V.last_error()
    need = V.rms_norm_workspace_bytes(4, 64)

    def backward(h=P, g=2 * P, w=3 * P, rstd=4 * P, dr=5 * P, dx=6 * P, dw=7 * P, ws=8 * P):
        return V.load().mimo_rms_norm_backward(4, 64, h, F, g, F, w, rstd, dr, dx, dw, ws, need, None)

    for bad in (dict(dx=P + 4), dict(dx=2 * P - 1020), dict(dx=3 * P + 252), dict(dx=4 * P + 12), dict(dx=5 * P + 4), dict(dx=7 * P - 1020),
                dict(dw=P + 1020), dict(dw=2 * P + 4), dict(dw=3 * P + 4), dict(dw=4 * P - 252), dict(dw=5 * P + 1020), dict(dw=6 * P + 512)):
        assert backward(**bad) == V.MIMO_E_INVALID and "in part" in V.last_error(), bad
    for at in (P, P + 1008, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P + 512, 7 * P):
        assert backward(ws=at) == V.MIMO_E_INVALID and "workspace" in V.last_error(), at


def test_mlp_refuses_arrays_that_overlap_in_part():
    """x, out, dout and dx are 512 bytes, the weights 9216, gate's and up's
    biases 288 and down's 256, hidden 1024, gate_up 4096."""
    lib = V.load()
    need = V.gated_mlp_workspace_bytes(4, 64, 72)

    def forward(out=10 * P, ws=20 * P, **kw):
        return lib.mimo_gated_mlp(_mlp(**kw), out, ws, need, None)

    for bad in (dict(out=P + 496), dict(out=2 * P + 9200), dict(out=3 * P - 496), dict(out=4 * P + 16), dict(out=5 * P + 272), dict(out=6 * P + 16),
                dict(out=7 * P + 240), dict(out=8 * P + 4080), dict(out=9 * P + 1008), dict(h=P + 16), dict(h=8 * P + 2048), dict(gu=4 * P - 16),
                dict(gu=9 * P - 4080), dict(gu=7 * P + 240)):
        assert forward(**bad) == V.MIMO_E_INVALID and "in part" in V.last_error(), bad
    for at in (P, 2 * P + 9200, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P + 240, 8 * P, 9 * P, 10 * P + 496, 10 * P - need + 16):
        assert forward(ws=at) == V.MIMO_E_INVALID and "workspace" in V.last_error(), at
    need = V.gated_mlp_backward_workspace_bytes(4, 64, 72)

    def backward(args=None, ws=20 * P, **kw):
        return lib.mimo_gated_mlp_backward(_mlp(**(args or {})), _mlp_grads(**kw), ws, need, None)

    for bad in (dict(dx=P + 496), dict(dx=11 * P - 496), dict(dx=13 * P + 9200), dict(dwg=2 * P + 9200), dict(dwu=3 * P - 16), dict(dwd=4 * P + 16),
                dict(dwd=9 * P + 1008), dict(dwg=8 * P + 4080), dict(dbg=16 * P + 4, dbu=16 * P), dict(dbu=12 * P + 508), dict(dbd=15 * P + 9212),
                dict(dbd=11 * P + 4)):
        assert backward(**bad) == V.MIMO_E_INVALID and "in part" in V.last_error(), bad
    for at in (P, 2 * P, 3 * P, 4 * P, 8 * P, 9 * P, 11 * P, 12 * P, 13 * P + 9200, 14 * P, 15 * P, 16 * P, 17 * P, 18 * P + 240, 18 * P - need + 16):
        assert backward(ws=at) == V.MIMO_E_INVALID and "workspace" in V.last_error(), at
