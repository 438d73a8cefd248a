"""GPU parity of the root-mean-square norm with the residual, forward, to 8-bit
rows and backward, against the float64 form on the same inputs.

Bars, derived from the arithmetic (e = 2^-24; u = 2^-8 for bf16 results, e for
float32).  A row of n values is summed by at least 64 threads, each in turn
over its own, then in a tree of 8 levels: a sum is off by at most D e times
the sum of magnitudes, D = n / 64 + 20.
  h:    the float32 sum, rounded to the residual's type: bit for bit
  rstd, relative: R = D e / 2 + 8 e (squares are positive; division, square
        root and reciprocal a few e)
  out:  (R + 3 e + u) |out|
  hat:  H = |hat| (R + e);  s = mean g hat: mean |g| H + (D + 3) e mean|g hat|
  dx:   rstd (3 e (|g| + |hat s|) + |hat| bar of s + H |s| + R |g - hat s|) + (e + u) |dx|
  dweight: sum |dout| H + (rows + 8) e sum |dout hat|
(1.01 covers products of two small terms.)  8-bit rows and their scales equal
the definition's.
"""
import numpy as np
import pytest

from oracle import tower

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
ROUND = {torch.float32: EPS, torch.bfloat16: 2.0 ** -8}
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}
NORM_EPS = 1e-6


def _say(*a):
    print("[gpu-rms]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _inputs(rows, width, x_kind, r_kind, g_kind, affine, seed):
    """x, residual (None without r_kind), dout, dresidual (of h's type), weight."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g)
    x = draw(rows, width).to(KIND[x_kind])
    res = (2 * draw(rows, width) + 0.5 * draw(width)).to(KIND[r_kind]) if r_kind else None
    dout = draw(rows, width).to(KIND[g_kind])
    dres = draw(rows, width).to(KIND[r_kind or x_kind])
    return x, res, dout, dres, 1 + 0.3 * draw(width) if affine else None


def _wide(t):
    return None if t is None else t.double().cpu().numpy()


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _within(got, want, bar, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    bad = err > 1.01 * bar + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float((err / (bar + 1e-30)).max()))


def _bars(r, dout, rows, n):
    """Bars of rstd (relative), out (relative, without its rounding), dx (without its rounding) and dweight."""
    depth = n / 64 + 20
    rel = depth * EPS / 2 + 8 * EPS
    hat, g, s = np.abs(r["hat"]), np.abs(r["g"]), np.abs(r["s"])[:, None]
    hat_bar = hat * (rel + EPS)
    s_bar = (g * hat_bar).mean(axis=1)[:, None] + (depth + 3) * EPS * (g * hat).mean(axis=1)[:, None]
    inner = np.abs(r["g"] - r["hat"] * r["s"][:, None])
    dx = r["rstd"][:, None] * (3 * EPS * (g + hat * s) + hat * s_bar + hat_bar * s + rel * inner) + EPS * np.abs(r["dx"])
    dw = (np.abs(dout) * hat_bar).sum(axis=0) + (rows + 8) * EPS * np.abs(dout * r["hat"]).sum(axis=0)
    return rel, rel + 3 * EPS, dx, dw


def _h(x, res):
    return x if res is None else (x.float() + res.float()).to(res.dtype)


def _check(V, rows, width, x_kind, r_kind, o_kind, g_kind, affine, seed, dres_too=True):
    _say((rows, width), x_kind, r_kind, o_kind, g_kind, "affine" if affine else "plain")
    x, res, dout, dres, w = _inputs(rows, width, x_kind, r_kind, g_kind, affine, seed)
    dres = dres if dres_too else None
    h = _h(x, res)
    if res is not None:
        assert np.array_equal(_wide(h), tower.residual_sum(_wide(x), _wide(res), r_kind))
    r = tower.rms_norm(_wide(h), _wide(w), NORM_EPS, _wide(dout), _wide(dres))
    rel, out_rel, dx_bar, dw_bar = _bars(r, _wide(dout), rows, width)
    xd, rd, gd, dd, wd = _dev(x, res, dout, dres, w)
    got = V.rms_norm(xd, wd, rd, eps=NORM_EPS, out_dtype=o_kind, return_rstd=True)
    hd = xd if res is None else got[1]
    dx, dw = V.rms_norm_backward(gd, hd, got[-1], wd, dresidual=dd, affine=True)
    q8 = V.rms_norm_quantized(xd, wd, rd, eps=NORM_EPS)
    torch.cuda.synchronize()
    assert len(got) == (2 if res is None else 3) and len(q8) == len(got)
    assert got[0].dtype == KIND[o_kind] and dx.dtype == h.dtype
    if res is not None:
        assert torch.equal(got[1].cpu(), h) and torch.equal(q8[2].cpu(), h)
    _within(got[-1], r["rstd"], rel * r["rstd"], "rstd")
    _within(got[0], r["out"], (out_rel + ROUND[KIND[o_kind]]) * np.abs(r["out"]), "out")
    _within(dx, r["dx"], dx_bar + ROUND[dx.dtype] * np.abs(r["dx"]), "dx")
    _within(dw, r["dweight"], dw_bar + EPS * np.abs(r["dweight"]), "dweight")
    q, scale = tower.rms_norm_quantized(_wide(h), _wide(w), NORM_EPS)
    assert np.array_equal(q8[1].cpu().numpy(), scale)
    assert np.array_equal(q8[0][:, :width].cpu().numpy(), q) and not q8[0][:, width:].any()
    assert q8[0].shape[1] % 128 == 0 and q8[0].shape[1] - width < 128


WIDTHS = [1, 2, 7, 8, 63, 64, 255, 256, 257, 512, 520, 1280, 1283, 1536, 1544, 2048, 2049, 4104, 5120, 6145, 8191, 16384, 16392, 20001]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_widths(V, width, kind):
    _check(V, 11, width, kind, kind, kind, kind, True, seed=width)


@pytest.mark.parametrize("x_kind,r_kind", [("f32", None), ("bf16", None), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("o_kind", ["f32", "bf16"])
@pytest.mark.parametrize("g_kind", ["f32", "bf16"])
def test_types(V, x_kind, r_kind, o_kind, g_kind):
    for width in (1280, 333, 5120, 16400):
        _check(V, 37, width, x_kind, r_kind, o_kind, g_kind, width != 333, seed=3, dres_too=o_kind == "f32")


@pytest.mark.parametrize("width", [504, 509, 1288, 1283, 2040, 2041, 5128, 5121, 8200, 8193, 16384, 16383])
@pytest.mark.parametrize("x_kind,r_kind,o_kind,g_kind", [("bf16", "f32", "f32", "f32"), ("bf16", "f32", "bf16", "bf16"),
                                                         ("bf16", "bf16", "f32", "f32"), ("f32", "f32", "bf16", "bf16")])
def test_mixed_types_in_every_shape(V, width, x_kind, r_kind, o_kind, g_kind):
    _check(V, 9, width, x_kind, r_kind, o_kind, g_kind, True, seed=width)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 1023, 1025, 4097, 9001])
def test_rows(V, rows):
    _check(V, rows, 72, "bf16", "bf16", "bf16", "bf16", True, seed=rows)
    _check(V, rows, 37, "f32", None, "f32", "f32", True, seed=rows + 1)


@pytest.mark.parametrize("rows,width", [(9001, 72), (9001, 509), (2500, 1280), (2500, 1283), (2500, 2041), (1700, 5120),
                                        (1700, 5121), (700, 8193), (700, 16384), (600, 20001)])
def test_workgroups_that_take_several_rows(V, rows, width):
    """More than twice as many rows as workgroups, in every shape: a sum has
    all of its rows, each once, and the same bits again."""
    _say("several rows a workgroup", (rows, width))
    groups = V.rms_norm_workspace_bytes(rows, width) // (4 * width)
    assert rows > 2 * groups > 0
    x, _, dout, _, w = _inputs(rows, width, "bf16", None, "f32", True, rows + width)
    r = tower.rms_norm(_wide(x), _wide(w), NORM_EPS, _wide(dout))
    xd, gd, wd = _dev(x, dout, w)
    _, rstd = V.rms_norm(xd, wd, eps=NORM_EPS, return_rstd=True)
    dx, dw = V.rms_norm_backward(gd, xd, rstd, wd)
    # additions on a value's way: over its workgroup's rows (or a wave's, and
    # then four waves), over the workgroups' sums of one of 32 threads, up their tree
    depth = -(-rows // groups) + -(-groups // 32) + 8 + 2 + 5
    _, _, dx_bar, _ = _bars(r, _wide(dout), rows, width)
    hat_bar = np.abs(r["hat"]) * ((width / 64 + 20) * EPS / 2 + 9 * EPS)
    dw_bar = (np.abs(_wide(dout)) * hat_bar).sum(axis=0) + depth * EPS * np.abs(_wide(dout) * r["hat"]).sum(axis=0)
    # no row's part of a sum is lost in the bar
    assert np.median(dw_bar) < np.median(np.abs(_wide(dout) * r["hat"])) / 4
    _within(dx, r["dx"], dx_bar + ROUND[dx.dtype] * np.abs(r["dx"]), "dx")
    _within(dw, r["dweight"], dw_bar + EPS * np.abs(r["dweight"]), "dweight")
    again = V.rms_norm_backward(gd, xd, rstd, wd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_gradient_against_differences(V):
    """The gradient along a direction against the difference of a loss in
    float64 at the kernel's own float32 outputs: off by the outputs' roundings
    over the step, and by the step squared."""
    _say("differences")
    rows, width, step = 5, 200, 2.0 ** -6
    x, res, dout, _, w = _inputs(rows, width, "f32", "f32", "f32", True, 77)
    way = torch.randn((rows, width), generator=torch.Generator().manual_seed(78))
    # values and steps on a grid that float32 sums hold exactly
    x, res, way = ((t * 2 ** 12).round() / 2 ** 12 for t in (x, res, way))
    wd, gd = w.cuda(), dout.cuda()

    def loss(s):
        return float((V.rms_norm((x + s * way).cuda(), wd, res.cuda(), eps=NORM_EPS)[0].double() * gd.double()).sum())

    out, h, rstd = V.rms_norm(x.cuda(), wd, res.cuda(), eps=NORM_EPS, return_rstd=True)
    dx, _ = V.rms_norm_backward(gd, h, rstd, wd)
    slope = float((dx.double().cpu() * way.double()).sum())
    mag = float((out.double().abs() * gd.double().abs()).sum())
    # the third derivative of h rstd along a way of about h's length is a few times its value
    bar = 2 * (width / 64 + 40) * EPS * mag / step + 16 * step ** 2 * mag
    assert abs((loss(step) - loss(-step)) / (2 * step) - slope) <= bar and bar < abs(slope)


def test_addresses_that_are_not_aligned(V):
    """The same rows one value further: other loads, the same bits."""
    _say("unaligned")
    for kind in ("f32", "bf16"):
        x, res, dout, dres, w = _dev(*_inputs(6, 1280, kind, kind, kind, True, 9))

        def shifted(t):
            s = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
            s.copy_(t)
            return s

        out, h, rstd = V.rms_norm(x, w, res, eps=NORM_EPS, return_rstd=True)
        o2, h2, r2 = V.rms_norm(shifted(x), shifted(w), shifted(res), eps=NORM_EPS, out=shifted(x), residual_out=shifted(x),
                                return_rstd=True)
        assert torch.equal(out, o2) and torch.equal(h, h2) and torch.equal(rstd, r2)
        q, s, _ = V.rms_norm_quantized(x, w, res)
        q2, s2, _ = V.rms_norm_quantized(shifted(x), shifted(w), shifted(res), residual_out=shifted(x))
        assert torch.equal(q, q2) and torch.equal(s, s2)
        dx, dw = V.rms_norm_backward(dout, h, rstd, w, dresidual=dres)
        dx2, dw2 = V.rms_norm_backward(shifted(dout), shifted(h), rstd, shifted(w), dresidual=shifted(dres), dx=shifted(dx))
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("width", [1280, 1283, 20001])
def test_in_place(V, width):
    """The stream updated in place, out over x, dx over dresidual: the same bits."""
    _say("in place", width)
    x, res, dout, dres, w = _dev(*_inputs(9, width, "bf16", "bf16", "bf16", True, 12))
    out, h, rstd = V.rms_norm(x, w, res, return_rstd=True)
    x2, r2 = x.clone(), res.clone()
    got = V.rms_norm(x2, w, r2, out=x2, residual_out=r2)
    assert got[0] is x2 and got[1] is r2 and torch.equal(x2, out) and torch.equal(r2, h)
    x2, r2 = x.clone(), res.clone()
    V.rms_norm(x2, w, r2, out=r2, residual_out=x2)
    assert torch.equal(r2, out) and torch.equal(x2, h)
    q, s, _ = V.rms_norm_quantized(x, w, res)
    r2 = res.clone()
    q2, s2, _ = V.rms_norm_quantized(x, w, r2, residual_out=r2)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(r2, h)
    dx, dw = V.rms_norm_backward(dout, h, rstd, w, dresidual=dres)
    d2 = dres.clone()
    assert V.rms_norm_backward(dout, h, rstd, w, dresidual=d2, dx=d2)[0] is d2 and torch.equal(d2, dx)
    assert V.rms_norm_backward(dout, h, rstd, w, affine=False)[1] is None


def test_rows_of_zeros_and_not_finite(V):
    _say("zeros, not finite")
    for width in (1280, 1283, 17000):
        x = torch.randn((6, width), generator=torch.Generator().manual_seed(4)).cuda()
        x[1] = 0
        x[2, 7] = float("nan")
        x[3, 9] = float("inf")
        x[4] = 1e-42
        out = V.rms_norm(x)
        assert (out[1] == 0).all() and torch.isnan(out[2]).all() and torch.isnan(out[3, 9]) and torch.isfinite(out[[0, 1, 4, 5]]).all()
        q, s = V.rms_norm_quantized(x)
        want_q, want_s = tower.rms_norm_quantized(_wide(x[[0, 1, 4, 5]]), None, 1e-6)
        assert np.array_equal(q[[0, 1, 4, 5], :width].cpu().numpy(), want_q) and np.array_equal(s[[0, 1, 4, 5]].cpu().numpy(), want_s)
        assert torch.isnan(s[2:4]).all() and not q[2:4].any() and s[1] == 0


def test_quantized_rows_go_into_the_product(V):
    """Norm to 8 bits and product, as a projection uses them, equal the norm in
    float32, its rows quantised, and the product, where no quotient is next to
    a border."""
    _say("norm and product")
    x, res, _, _, w = _dev(*_inputs(300, 1283, "bf16", "bf16", "bf16", True, 15))
    wq, ws = V.quantize_rows(torch.randn((640, 1283), generator=torch.Generator().manual_seed(16)).cuda())
    q, s, h = V.rms_norm_quantized(x, w, res)
    got = V.quantized_linear(q, s, wq, ws)
    ref, mag = tower.quantized_linear(q.cpu().numpy(), s.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy())
    _within(got, ref, (2.0 ** -8 + 4 * EPS) * np.abs(ref) + 4 * EPS * mag, "product")


def test_empty(V):
    _say("empty")
    x = torch.zeros((0, 1280), device="cuda")
    w = torch.ones(1280, device="cuda")
    out, h, rstd = V.rms_norm(x, w, x, return_rstd=True)
    assert out.shape == h.shape == (0, 1280) and rstd.shape == (0,)
    q, s = V.rms_norm_quantized(x, w)
    assert q.shape == (0, 1280) and s.shape == (0,)
    dx, dw = V.rms_norm_backward(x, x, rstd, w)
    assert dx.shape == (0, 1280) and (dw == 0).all()


def test_streams_and_graphs(V):
    _say("streams and graphs")
    mk = lambda s: _dev(*_inputs(300, 1280, "bf16", "bf16", "bf16", True, s))

    def step(x, res, dout, dres, w, stream=None):
        out, h, rstd = V.rms_norm(x, w, res, return_rstd=True, stream=stream)
        return (out, h, *V.rms_norm_quantized(x, w, res, stream=stream),
                *V.rms_norm_backward(dout, h, rstd, w, dresidual=dres, stream=stream))

    x = mk(20)
    want = step(*x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(*x, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held = []
    for seed in (21, 22):
        st = mk(seed)
        step(*st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*st)
        held.append((graph, st, outs))
    for turn in range(3):
        for i, (graph, st, outs) in enumerate(held):
            for t, new in zip(st, mk(30 + 2 * turn + i)):
                t.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, step(*st)):
                assert torch.equal(a, b)


def test_past_32_bits(V):
    """1.7 million rows: parts of a large call equal the same parts called alone."""
    _say("1.7 million rows")
    n, width = 1_700_003, 1280
    x = torch.empty((n, width), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for part in x.split(1 << 17):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    w = torch.rand(width, generator=torch.Generator().manual_seed(7)).cuda()
    out, h, rstd = V.rms_norm(x, w, x, return_rstd=True)
    q, s, _ = V.rms_norm_quantized(x, w, x, residual_out=h)
    dx, dw = V.rms_norm_backward(out, h, rstd, w, dresidual=x)
    for at in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        o, hh, r = V.rms_norm(x[at], w, x[at], return_rstd=True)
        assert torch.equal(o, out[at]) and torch.equal(hh, h[at]) and torch.equal(r, rstd[at])
        q1, s1, _ = V.rms_norm_quantized(x[at], w, x[at])
        assert torch.equal(q1, q[at]) and torch.equal(s1, s[at])
        assert torch.equal(V.rms_norm_backward(o, hh, r, w, dresidual=x[at])[0], dx[at])
    want = torch.zeros(width, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for i in range(0, n, 1 << 16):
        t = out[i:i + (1 << 16)].double() * h[i:i + (1 << 16)].double() * rstd[i:i + (1 << 16)].double()[:, None]
        want += t.sum(0)
        mag += t.abs().sum(0)
    # additions on a value's way, as above, and hat's rounding
    groups = V.rms_norm_workspace_bytes(n, width) // (4 * width)
    assert ((dw.double() - want).abs() <= (-(-n // groups) + groups // 32 + 20) * EPS * mag).all()


def test_refusals(V):
    _say("refusals")
    x = torch.zeros((4, 64), device="cuda")
    b = x.to(torch.bfloat16)
    w = torch.ones(64, device="cuda")
    r = torch.ones(4, device="cuda")
    for bad in (lambda: V.rms_norm(x.t()), lambda: V.rms_norm(x, w[:32]), lambda: V.rms_norm(x, w, b), lambda: V.rms_norm(x, w, x[:2]),
                lambda: V.rms_norm(x, w.cpu()), lambda: V.rms_norm(x, residual_out=x), lambda: V.rms_norm(x, out_dtype="f16"),
                lambda: V.rms_norm(x, eps=-1.0), lambda: V.rms_norm(x.half()), lambda: V.rms_norm(x, w, x, residual_out=b),
                lambda: V.rms_norm(b, w, x, out=x, residual_out=x), lambda: V.rms_norm(x, out=x[:2]),
                lambda: V.rms_norm(x, rstd=r[:2]), lambda: V.rms_norm_quantized(x, q=torch.zeros((4, 64), dtype=torch.int8, device="cuda")),
                lambda: V.rms_norm_quantized(x, scale=w), lambda: V.rms_norm_backward(x, x, None), lambda: V.rms_norm_backward(x[:2], x, r),
                lambda: V.rms_norm_backward(x, x, r, dresidual=b), lambda: V.rms_norm_backward(x, x, r, dx=x),
                lambda: V.rms_norm_backward(x, x, r, w, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")),
                lambda: V.rms_norm(torch.zeros((2, 65537), device="cuda"))):
        with pytest.raises(V.MimoError):
            bad()


@pytest.mark.parametrize("width", [8, 509, 1280, 1283, 5120, 8193, 16384, 20001])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-60])
def test_small_and_large_rows(V, width, eps):
    """Rows whose squares pass float32's range on either side, as eps allows
    them: rstd, out and the gradients are the formula's, and the 8-bit form's
    integers too.  The bars are relative, so they hold at any power of two that
    rstd and the gradients can be held at.  Gradients of the largest rows are
    not: below 2^-126 a type's steps stay what they are there, 2^-149 in float32
    and 2^-133 in bf16, and a rounding is off by half of one at most (the float64
    gradient rounded to bf16 alone is 3.8 of the relative bars away at width
    509, in the row of 2^120), so dx has these halves in its bar."""
    _say("small and large rows", width, eps)
    x, _, dout, _, w = _inputs(12, width, "f32", None, "f32", True, seed=width)
    powers = [-120, -110, -100, -80, -70, -60, -50, 0, 60, 70, 100, 120]
    x = x * torch.tensor([2.0 ** p for p in powers])[:, None]
    for kind in ("f32", "bf16"):
        xk, gk = x.to(KIND[kind]), dout.to(KIND[kind])
        r = tower.rms_norm(_wide(xk), _wide(w), eps, _wide(gk))
        xd, gd, wd = _dev(xk, gk, w)
        rel, out_rel, dx_bar, dw_bar = _bars(r, _wide(gk), 12, width)
        out, rstd = V.rms_norm(xd, wd, eps=eps, return_rstd=True)
        assert (np.abs(_wide(rstd) / r["rstd"] - 1) <= rel + EPS).all()
        _within(out, r["out"], (out_rel + ROUND[xk.dtype]) * np.abs(r["out"]), "out")
        # with a residual of zeros the sum is x, and a float32 stream's rows go the same way
        two = V.rms_norm(xd, wd, torch.zeros_like(xd, dtype=torch.float32), eps=eps, out_dtype="f32", return_rstd=True)
        assert torch.equal(two[1], xd.float()) and torch.equal(two[2], rstd)
        dx, dw = V.rms_norm_backward(gd, xd, rstd, wd)
        unit = 1 / r["rstd"][:, None]  # a row's gradients next to one
        step = 2.0 ** -150 + (2.0 ** -134 if kind == "bf16" else 0.0)
        _within(dx.double().cpu() * torch.from_numpy(unit), r["dx"] * unit, (dx_bar + ROUND[dx.dtype] * np.abs(r["dx"]) + step) * unit, "dx")
        _within(dw, r["dweight"], dw_bar + EPS * np.abs(r["dweight"]), "dweight")
        q, scale = tower.rms_norm_quantized(_wide(xk), _wide(w), eps)
        got_q, got_scale = V.rms_norm_quantized(xd, wd, eps=eps)
        assert np.array_equal(got_q[:, :width].cpu().numpy(), q) and np.array_equal(got_scale.cpu().numpy(), scale)


def test_quantized_norm_and_product_from_its_definition(V):
    """Norm to 8 bits and product, as a projection uses them, from the
    definition's integers and scales of the rounded sum; and next to the norm in
    float32 whose rows are quantised by a call of their own, whose rstd may
    differ in its last bits: no integer is more than one away, and only those
    whose quotient lies next to the middle of two are."""
    _say("norm, integers and product")
    x, res, _, _, w = _inputs(300, 1283, "bf16", "bf16", "bf16", True, 15)
    xd, rd, wd = _dev(x, res, w)
    wq, ws = V.quantize_rows(torch.randn((640, 1283), generator=torch.Generator().manual_seed(16)).cuda())
    got = V.quantized_linear(*V.rms_norm_quantized(xd, wd, rd)[:2], wq, ws)
    q, s = tower.rms_norm_quantized(_wide(_h(x, res)), _wide(w), 1e-6)
    padded = np.zeros((300, wq.shape[1]), dtype=np.int8)
    padded[:, :1283] = q
    ref, mag = tower.quantized_linear(padded, s, wq.cpu().numpy(), ws.cpu().numpy())
    _within(got, ref, (2.0 ** -8 + 4 * EPS) * np.abs(ref) + 4 * EPS * mag, "product")
    y = V.rms_norm(xd, wd, rd, out_dtype="f32")[0]
    q2, s2 = V.quantize_rows(y)
    r = tower.rms_norm(_wide(_h(x, res)), _wide(w), 1e-6)["out"]
    # relative to a value: rstd's bar and the products' roundings of both forms; a scale's holds the division's too
    rel = 2 * ((1283 / 64 + 20) * EPS / 2 + 12 * EPS)
    assert (np.abs(_wide(s2) - s.astype(np.float64)) <= rel * s).all()
    apart = np.abs(q2[:, :1283].cpu().numpy().astype(int) - q.astype(int))
    quotient = np.abs(r) / s.astype(np.float64)[:, None]
    middle = np.abs(quotient - np.floor(quotient) - 0.5)
    assert apart.max() <= 1 and (middle[apart > 0] <= 2 * rel * 128).all() and not q2[:, 1283:].any()


def test_partial_sums_are_added_in_more_than_float32(V):
    """256 rows over 256 workgroups, every partial sum one row's, exactly: the
    weight's gradient is the sum rounded once, although a float32 one would lose
    each 1 that is added to 2^24."""
    _say("partial sums")
    width = 1280
    assert V.rms_norm_workspace_bytes(256, width) == 256 * width * 4
    x = torch.ones((256, width), device="cuda")
    dout = torch.ones((256, width), device="cuda")
    dout[torch.arange(width) % 256, torch.arange(width)] = 2.0 ** 24
    _, rstd = V.rms_norm(x, eps=0.0, return_rstd=True)
    assert (rstd == 1).all()
    dw = V.rms_norm_backward(dout, x, rstd, affine=True)[1]
    assert torch.equal(dw, dout.double().sum(0).float()) and (dw == 2.0 ** 24 + 256).all()
