"""GPU parity of layer norm, forward and backward, against the float64 form on
the same inputs.

Bars, derived from the arithmetic (e = 2^-24; u = 2^-8 for bf16 results, e for
float32).  A row of n values is summed by at least 64 threads, each in turn
over its own, then in a tree of 8 levels: a sum is off by at most D e times
the sum of magnitudes, D = n / 64 + 20.
  mean: M = D e mean|x|;  rstd, relative: R = (D + 8) e + M^2 rstd^2 + 4 e
  hat:  H = rstd (M + 2 e |x - mean|) + |hat| R
  out:  |w| H + 3 e (|hat w| + |b|) + u |out|
  s1 = mean g: D e mean|g|;   s2 = mean g hat: mean |g| H + (D + 2) e mean|g hat|
  dx:   rstd (4 e (|g| + |s1| + |hat s2|) + bars of s1 and of s2 times |hat| + H |s2|) + R |dx| + u |dx|
  dweight: sum |dout| H + (rows + 8) e sum |dout hat|;  dbias: (rows + 8) e sum |dout|
(1.01 covers products of two small terms.)
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
    print("[gpu-norm]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _inputs(rows, width, x_kind, g_kind, affine, seed, offset=0.5, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, width), generator=g) * spread + offset * torch.randn(width, generator=g)).to(KIND[x_kind])
    dout = torch.randn((rows, width), generator=g).to(KIND[g_kind])
    w = 1 + 0.3 * torch.randn(width, generator=g) if affine else None
    b = 0.3 * torch.randn(width, generator=g) if affine else None
    return x, dout, w, b


def _wide(t):
    return None if t is None else t.double().cpu().numpy()


def _within(got, want, bar, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    bad = err > 1.01 * bar + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float((err / (bar + 1e-30)).max()))


def _bars(x, dout, w, b, r, eps_norm=NORM_EPS):
    rows, n = x.shape
    depth = n / 64 + 20
    mean = (depth * EPS * np.abs(x).mean(axis=1))[:, None]
    rstd = r["rstd"][:, None]
    rel = (depth + 8) * EPS + mean ** 2 * rstd ** 2 + 4 * EPS
    hat = rstd * (mean + 2 * EPS * np.abs(x - r["mean"][:, None])) + np.abs(r["hat"]) * rel
    w1 = np.ones(n) if w is None else np.abs(w)
    out = w1 * hat + 3 * EPS * (np.abs(r["hat"]) * w1 + (0 if b is None else np.abs(b)))
    if dout is None:
        return mean[:, 0], rel[:, 0], out
    g, s1, s2 = np.abs(r["g"]), np.abs(r["s1"])[:, None], np.abs(r["s2"])[:, None]
    s1_bar = (depth * EPS * g.mean(axis=1))[:, None]
    s2_bar = (g * hat).mean(axis=1)[:, None] + (depth + 2) * EPS * (g * np.abs(r["hat"])).mean(axis=1)[:, None]
    dx = rstd * (4 * EPS * (g + s1 + np.abs(r["hat"]) * s2) + s1_bar + np.abs(r["hat"]) * s2_bar + hat * s2) + rel * np.abs(r["dx"])
    dw = (np.abs(dout) * hat).sum(axis=0) + (rows + 8) * EPS * np.abs(dout * r["hat"]).sum(axis=0)
    db = (rows + 8) * EPS * np.abs(dout).sum(axis=0)
    return mean[:, 0], rel[:, 0], out, dx, dw, db


def _check(V, rows, width, x_kind, o_kind, g_kind, affine, seed, **kw):
    _say((rows, width), x_kind, o_kind, g_kind, "affine" if affine else "plain")
    x, dout, w, b = _inputs(rows, width, x_kind, g_kind, affine, seed, **kw)
    r = tower.layer_norm(_wide(x), _wide(w), _wide(b), NORM_EPS, _wide(dout))
    mean_bar, rel, out_bar, dx_bar, dw_bar, db_bar = _bars(_wide(x), _wide(dout), _wide(w), _wide(b), r)
    dev = [None if t is None else t.cuda() for t in (x, dout, w, b)]
    out, mean, rstd = V.layer_norm(dev[0], dev[2], dev[3], eps=NORM_EPS, out_dtype=o_kind, return_stats=True)
    dx, dw, db = V.layer_norm_backward(dev[1], dev[0], mean, rstd, dev[2], affine=True)
    torch.cuda.synchronize()
    assert out.dtype == KIND[o_kind] and dx.dtype == x.dtype
    _within(mean, r["mean"], mean_bar + EPS * np.abs(r["mean"]), "mean")
    _within(rstd, r["rstd"], rel * r["rstd"], "rstd")
    _within(out, r["out"], out_bar + ROUND[out.dtype] * np.abs(r["out"]), "out")
    _within(dx, r["dx"], dx_bar + ROUND[dx.dtype] * np.abs(r["dx"]), "dx")
    _within(dw, r["dweight"], dw_bar + EPS * np.abs(r["dweight"]), "dweight")
    _within(db, r["dbias"], db_bar + EPS * np.abs(r["dbias"]), "dbias")


@pytest.mark.parametrize("width", [1, 2, 7, 8, 63, 64, 255, 256, 257, 512, 520, 1280, 1283, 1536, 1544, 2048, 2049, 4096,
                                   4104, 5120, 8191, 8193, 16384, 16392, 20001])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_widths(V, width, kind):
    _check(V, 11, width, kind, kind, kind, True, seed=width)


@pytest.mark.parametrize("x_kind", ["f32", "bf16"])
@pytest.mark.parametrize("o_kind", ["f32", "bf16"])
@pytest.mark.parametrize("g_kind", ["f32", "bf16"])
@pytest.mark.parametrize("affine", [True, False])
def test_types(V, x_kind, o_kind, g_kind, affine):
    for width in (1280, 333, 5120):
        _check(V, 37, width, x_kind, o_kind, g_kind, affine, seed=3)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 1023, 1025, 4097, 9001])
def test_rows(V, rows):
    _check(V, rows, 72, "bf16", "bf16", "bf16", True, seed=rows)
    _check(V, rows, 37, "f32", "f32", "f32", True, seed=rows + 1)


def _sums_depth(V, rows, width):
    """(workgroups, additions on a value's way into dweight or dbias): over the
    rows of its workgroup (or of a wave, and then four waves), over the
    workgroups' sums that one of the last launch's 32 threads a column takes,
    and up their tree; and eight to spare."""
    groups = V.layer_norm_workspace_bytes(rows, width) // (2 * 4 * width)
    assert groups > 0
    return groups, -(-rows // groups) + -(-groups // 32) + 8 + 2 + 5


@pytest.mark.parametrize("rows,width", [(9001, 72), (9001, 509), (2500, 1280), (2500, 1283), (2500, 2041), (1700, 5120),
                                        (1700, 5121), (700, 8192), (700, 8193), (700, 16384), (700, 16392), (600, 20001)])
@pytest.mark.parametrize("x_kind,g_kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_workgroups_that_take_several_rows(V, rows, width, x_kind, g_kind):
    """More than twice as many rows as workgroups, in every shape, aligned and
    not: a sum has all of its rows, each once."""
    _say("several rows a workgroup", (rows, width), x_kind, g_kind)
    groups, depth = _sums_depth(V, rows, width)
    assert rows > 2 * groups
    x, dout, w, b = _inputs(rows, width, x_kind, g_kind, True, rows + width)
    wide = [_wide(t) for t in (x, dout, w, b)]
    r = tower.layer_norm(wide[0], wide[2], wide[3], NORM_EPS, wide[1])
    mean_bar, rel, _, dx_bar, _, _ = _bars(*wide, r)
    dev = [t.cuda() for t in (x, dout, w, b)]
    _, mean, rstd = V.layer_norm(dev[0], dev[2], dev[3], eps=NORM_EPS, return_stats=True)
    dx, dw, db = V.layer_norm_backward(dev[1], dev[0], mean, rstd, dev[2])
    _within(dx, r["dx"], dx_bar + ROUND[dx.dtype] * np.abs(r["dx"]), "dx")
    hat = r["rstd"][:, None] * (mean_bar[:, None] + 2 * EPS * np.abs(wide[0] - r["mean"][:, None])) + np.abs(r["hat"]) * rel[:, None]
    dw_bar = (np.abs(wide[1]) * hat).sum(axis=0) + depth * EPS * np.abs(wide[1] * r["hat"]).sum(axis=0)
    db_bar = depth * EPS * np.abs(wide[1]).sum(axis=0)
    # no row's part of a sum is lost in the bar
    assert np.median(dw_bar) < np.median(np.abs(wide[1] * r["hat"])) / 4 and np.median(db_bar) < np.median(np.abs(wide[1])) / 4
    _within(dw, r["dweight"], dw_bar + EPS * np.abs(r["dweight"]), "dweight")
    _within(db, r["dbias"], db_bar + EPS * np.abs(r["dbias"]), "dbias")
    again = V.layer_norm_backward(dev[1], dev[0], mean, rstd, dev[2])
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


def test_large_mean(V):
    """A mean a thousand times the spread: the variance is taken from the
    distances, not from a difference of large numbers."""
    _check(V, 40, 1280, "f32", "f32", "f32", True, seed=5, offset=1000.0, spread=1.0)


def test_addresses_that_are_not_aligned(V):
    """The same rows one value further: other loads, the same bars."""
    _say("unaligned")
    for kind in ("f32", "bf16"):
        x, dout, w, b = _inputs(6, 1280, kind, kind, True, 9)
        r = tower.layer_norm(_wide(x), _wide(w), _wide(b), NORM_EPS, _wide(dout))
        _, _, out_bar, dx_bar, dw_bar, db_bar = _bars(_wide(x), _wide(dout), _wide(w), _wide(b), r)

        def shifted(t):
            s = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
            s.copy_(t)
            return s

        xs, gs, ws, bs = shifted(x), shifted(dout), shifted(w), shifted(b)
        out, mean, rstd = V.layer_norm(xs, ws, bs, eps=NORM_EPS, out=shifted(x), return_stats=True)
        dx, dw, db = V.layer_norm_backward(gs, xs, mean, rstd, ws, dx=shifted(x))
        _within(out, r["out"], out_bar + ROUND[out.dtype] * np.abs(r["out"]), "out")
        _within(dx, r["dx"], dx_bar + ROUND[dx.dtype] * np.abs(r["dx"]), "dx")
        _within(dw, r["dweight"], dw_bar + EPS * np.abs(r["dweight"]), "dweight")
        _within(db, r["dbias"], db_bar + EPS * np.abs(r["dbias"]), "dbias")


def test_rows_of_equal_values_and_not_finite(V):
    _say("equal values, not finite")
    x = torch.full((4, 1280), 3.25, device="cuda")
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    b = torch.arange(1280.0, device="cuda")
    out, mean, rstd = V.layer_norm(x, None, b, return_stats=True)
    assert torch.equal(out[0], b) and torch.equal(out[3], b) and torch.isnan(out[1:3]).all()
    assert rstd[0].item() == pytest.approx(1000.0, rel=1e-6)


def test_in_place_units_and_parts(V):
    """out = x; merge units as a view; sums of one parameter alone."""
    _say("in place, units, parts")
    x, dout, w, b = (t.cuda() for t in _inputs(64, 1280, "bf16", "bf16", True, 12))
    want, mean, rstd = V.layer_norm(x, w, b, return_stats=True)
    y = x.clone()
    assert V.layer_norm(y, w, b, out=y) is y and torch.equal(y, want)
    units = V.layer_norm(x.view(16, 5120))
    r = tower.layer_norm(_wide(x.view(16, 5120)), None, None, NORM_EPS)
    _, _, out_bar = _bars(_wide(x.view(16, 5120)), None, None, None, r)
    _within(units, r["out"], out_bar + ROUND[units.dtype] * np.abs(r["out"]), "units")
    dx, dw, db = V.layer_norm_backward(dout, x, mean, rstd, w)
    only = torch.full((1280,), 5.0, device="cuda")
    dx2, none, got = V.layer_norm_backward(dout, x, mean, rstd, w, dbias=only, affine=False)
    assert none is None and got is only and torch.equal(only, db) and torch.equal(dx2, dx)
    dx3, a, b2 = V.layer_norm_backward(dout, x, mean, rstd, w, affine=False)
    assert a is None and b2 is None and torch.equal(dx3, dx)


def test_empty(V):
    _say("empty")
    x = torch.zeros((0, 1280), device="cuda")
    w = torch.ones(1280, device="cuda")
    out, mean, rstd = V.layer_norm(x, w, w, return_stats=True)
    assert out.shape == (0, 1280) and mean.shape == (0,)
    dx, dw, db = V.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 1280) and (dw == 0).all() and (db == 0).all()


def test_streams_and_graphs(V):
    _say("streams and graphs")
    mk = lambda s: [t.cuda() for t in _inputs(300, 1280, "bf16", "bf16", True, s)]

    def step(x, dout, w, b, stream=None):
        out, mean, rstd = V.layer_norm(x, w, b, return_stats=True, stream=stream)
        return (out, *V.layer_norm_backward(dout, x, mean, rstd, w, stream=stream))

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
