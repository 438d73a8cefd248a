"""GPU parity of the gated feed-forward block, forward and backward, against
the float64 form on the same inputs.

Bars, derived from the arithmetic (e = 2^-24 float32, v = 2^-8 bf16).  A sum of
K products of bf16 values is off by at most (K + 8) e times the sum of their
magnitudes, whatever its order.  |silu'| <= 1.1 and |silu''| <= 0.5 everywhere,
and g^2 s (1 - s) < 1, so the exponential's rounding (2 e |g| relative) moves
silu by 2 e at most.
  g:  G = (D + 8) e (sum |x||wg| + |bg|);  u: U, the same
  silu: A = 1.1 G + 8 e |silu| + 2 e
  h:  |u| A + |silu| U + A U + 4 e |h|, and its rounding v |h|
  out: sum (bar of h) |wd| + (H + 8) e (sum |h||wd| + |bd|) + v |out|
  dh: (D + 8) e sum |dout||wd|
  dg: |u silu'| bar(dh) + |dh silu'| U + |dh u| (0.5 G + 12 e) + 4 e |dg|; as an operand, and v |dg|
  du: |silu| bar(dh) + |dh| A + 4 e |du|; as an operand, and v |du|
  dx: sums of the operands' bars + (2 H + 8) e times the sum of magnitudes + v |dx|
  weights: the same over rows, (rows + 8) e; biases: sums of the bars without v,
  (rows + 8) e times the sum of magnitudes, e |db|
(1.05 covers products of two small terms.)
"""
import numpy as np
import pytest

import mlp_tiles
from oracle import tower

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS, U8 = 2.0 ** -24, 2.0 ** -8
GRADS = ("dx", "dw_gate", "dw_up", "dw_down", "db_gate", "db_up", "db_down")


def _say(*a):
    print("[gpu-mlp]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _inputs(rows, d, h, bias, seed, scale=1.0):
    """x, the three weights, the three biases (None without), dout."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g)
    bf = lambda t: t.to(torch.bfloat16)
    x, dout = bf(draw(rows, d)), bf(draw(rows, d))
    w = bf(draw(h, d) * scale * d ** -0.5), bf(draw(h, d) * d ** -0.5), bf(draw(d, h) * h ** -0.5)
    b = tuple(0.2 * draw(n) for n in (h, h, d)) if bias else (None, None, None)
    return x, w, b, dout


def _wide(t):
    return None if t is None else t.double().cpu().numpy()


def _dev(t):
    return None if t is None else t.cuda()


def _within(got, want, bar, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all(), what
    err = np.abs(got - want)
    bad = err > 1.05 * bar + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float((err / (bar + 1e-30)).max()))


def _bars(x, w, b, dout, r):
    rows, d = x.shape
    h = w[0].shape[0]
    ax, aw = np.abs(x), [np.abs(t) for t in w]
    a = {k: np.abs(t) for k, t in r.items()}
    mag = lambda t: 0.0 if t is None else np.abs(t)
    G, U = ((d + 8) * EPS * (ax @ aw[i].T + mag(b[i])) for i in (0, 1))
    A = 1.1 * G + 8 * EPS * a["silu"] + 2 * EPS
    H = a["up"] * A + a["silu"] * U + A * U + 4 * EPS * a["hidden"]
    bars = {"gate": G, "up": U, "hidden": H + U8 * a["hidden"]}
    bars["out"] = bars["hidden"] @ aw[2].T + (h + 8) * EPS * (a["hidden"] @ aw[2].T + mag(b[2])) + U8 * a["out"]
    if dout is None:
        return bars
    ad = np.abs(dout)
    DH = (d + 8) * EPS * (ad @ aw[2])
    DG = a["up"] * a["slope"] * DH + a["dhidden"] * a["slope"] * U + a["dhidden"] * a["up"] * (0.5 * G + 12 * EPS) + 4 * EPS * a["dgate"]
    DU = a["silu"] * DH + a["dhidden"] * A + 4 * EPS * a["dup"]
    og, ou = DG + U8 * a["dgate"], DU + U8 * a["dup"]
    bars["dx"] = og @ aw[0] + ou @ aw[1] + (2 * h + 8) * EPS * (a["dgate"] @ aw[0] + a["dup"] @ aw[1]) + U8 * a["dx"]
    n = (rows + 8) * EPS
    bars["dw_gate"] = og.T @ ax + n * (a["dgate"].T @ ax) + U8 * a["dw_gate"]
    bars["dw_up"] = ou.T @ ax + n * (a["dup"].T @ ax) + U8 * a["dw_up"]
    bars["dw_down"] = ad.T @ bars["hidden"] + n * (ad.T @ a["hidden"]) + U8 * a["dw_down"]
    bars["db_gate"] = DG.sum(axis=0) + n * a["dgate"].sum(axis=0) + EPS * a["db_gate"]
    bars["db_up"] = DU.sum(axis=0) + n * a["dup"].sum(axis=0) + EPS * a["db_up"]
    bars["db_down"] = n * ad.sum(axis=0) + EPS * a["db_down"]
    return bars


def _poison(n):
    """A workspace of NaNs, whatever type is read from it."""
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")


def _check(V, rows, d, h, bias, seed, backward=True, scale=1.0):
    _say((rows, d, h), "bias" if bias else "no bias", "scale", scale)
    x, w, b, dout = _inputs(rows, d, h, bias, seed, scale)
    wide = _wide(x), [_wide(t) for t in w], [_wide(t) for t in b], _wide(dout) if backward else None
    r = tower.gated_mlp(wide[0], *wide[1], *wide[2], wide[3])
    bars = _bars(*wide, r)
    xd, gd, wd, bd = _dev(x), _dev(dout), [_dev(t) for t in w], [_dev(t) for t in b]
    ws = _poison(V.gated_mlp_workspace_bytes(rows, d, h))
    out, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True, workspace=ws, out=torch.full_like(xd, float("nan")))
    plain = V.gated_mlp(xd, *wd, *bd)
    torch.cuda.synchronize()
    _within(out, r["out"], bars["out"], "out")
    assert torch.equal(plain, out)
    padded = (h + 63) // 64 * 64
    assert gate_up.shape == (2, rows, padded) and hidden.shape == (rows, padded)
    _within(gate_up[0, :, :h], r["gate"], bars["gate"] + EPS * np.abs(r["gate"]), "gate")
    _within(gate_up[1, :, :h], r["up"], bars["up"] + EPS * np.abs(r["up"]), "up")
    _within(hidden[:, :h], r["hidden"], bars["hidden"], "hidden")
    assert not hidden[:, h:].any() and not gate_up[:, :, h:].any()
    if not backward:
        return
    ws = _poison(V.gated_mlp_backward_workspace_bytes(rows, d, h))
    got = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True, workspace=ws)
    torch.cuda.synchronize()
    for name, t in zip(GRADS, got):
        _within(t, r[name], bars[name], name)
    again = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden)
    assert all(torch.equal(a, c) for a, c in zip(got[:4], again[:4])) and again[4:] == (None, None, None)


@pytest.mark.parametrize("rows,d,h", [(1, 1, 1), (1, 8, 8), (2, 7, 9), (1, 64, 64), (3, 72, 40), (4, 1280, 512), (16, 128, 192), (17, 136, 200),
                                      (32, 320, 64), (33, 64, 328), (63, 100, 100), (64, 1283, 131), (65, 129, 321), (100, 520, 264),
                                      (128, 128, 128), (129, 65, 130), (216, 640, 1000), (257, 263, 513), (700, 96, 1032), (1000, 1024, 72)])
@pytest.mark.parametrize("bias", [False, True])
def test_sizes(V, rows, d, h, bias):
    _check(V, rows, d, h, bias, rows + d + h)


@pytest.mark.parametrize("rows,d,h", [(4200, 136, 2056), (8300, 72, 2051), (16500, 1032, 80), (40, 4100, 4104), (1, 2000, 5000), (3, 5000, 2000),
                                      (9, 4099, 1283), (31, 1280, 5120), (32, 2048, 2048), (29, 1283, 3421),
                                      (29, 1283, 1027)])
def test_large(V, rows, d, h):
    """Every kernel's large tiles, long sums, and one row."""
    _check(V, rows, d, h, True, 7)


@pytest.mark.parametrize("rows,d,h", [(14394, 947, 967), (14394, 947, 968), (10955, 132, 3634), (19658, 194, 3313)])
def test_tiles_of_256(V, rows, d, h):
    """Sizes whose products go by tiles of 256 x 256, all of them, and those
    whose sums for out, dx and the weights' gradients are made in parts."""
    _check(V, rows, d, h, True, 3)


@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_gates_near_zero_and_saturated(V, scale):
    _check(V, 70, 96, 200, True, 11, scale=scale)


def test_far_gates(V):
    """Gates beyond exp's range in float32: silu is g or 0, its slope 1 or 0."""
    _say("far gates")
    x = torch.full((4, 8), 1.0).to(torch.bfloat16).cuda()
    x[1] = -1
    w = torch.full((8, 8), 200.0).to(torch.bfloat16).cuda()
    one = torch.full((8, 8), 0.125).to(torch.bfloat16).cuda()
    out, gate_up, hidden = V.gated_mlp(x, w, one, one, return_saved=True)
    assert (hidden[0, :8] == 1600).all() and (hidden[1, :8] == 0).all() and (out[0] == 1600).all()
    dx, *_ = V.gated_mlp_backward(x, x, w, one, one, gate_up, hidden)
    assert torch.isfinite(dx).all()


def test_rows_do_not_reach_others(V):
    """A row of NaN reaches its own outputs only, forward and in dx."""
    _say("NaN in one row")
    for rows in (40, 300):
        x, w, b, dout = _inputs(rows, 136, 200, True, 3)
        xd, wd, bd, gd = _dev(x), [_dev(t) for t in w], [_dev(t) for t in b], _dev(dout)
        want, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
        dx = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden)[0]
        xd[7] = float("nan")
        gd[9] = float("inf")
        out, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
        dx2 = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden)[0]
        keep = torch.arange(rows) != 7
        assert torch.equal(out[keep], want[keep]) and torch.isnan(out[7]).all()
        keep &= torch.arange(rows) != 9
        assert torch.equal(dx2[keep], dx[keep])


@pytest.mark.parametrize("rows,d,h", [(37, 64, 200), (1100, 1280, 1288), (14300, 944, 968)])
def test_infinities_of_the_last_row(V, rows, d, h):
    """An infinity of dout in the last row makes dg and du of that row infinite,
    and so the biases' gradients: with u's and silu's sign, not NaN from the
    rows behind the last one, which are none."""
    _say("infinities", (rows, d, h))
    x, w, _, dout = _inputs(rows, d, h, False, 5)
    xd, gd, wd = _dev(x), _dev(dout), [_dev(t) for t in w]
    wd[2] = wd[2].abs() + 2.0 ** -6
    gd[-1, 3] = float("inf")
    _, gate_up, hidden = V.gated_mlp(xd, *wd, return_saved=True)
    *_, db_gate, db_up, db_down = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True)
    g, u = (gate_up[i, -1, :h].double() for i in (0, 1))
    s = torch.sigmoid(g)
    inf = torch.full_like(g, float("inf"))
    assert torch.equal(db_gate.double(), torch.copysign(inf, u * s * (1 + g * (1 - s))))
    assert torch.equal(db_up.double(), torch.copysign(inf, g * s))
    assert db_down[3] == float("inf") and torch.isfinite(torch.cat([db_down[:3], db_down[4:]])).all()


def test_parts_of_the_gradients(V):
    """Only those that are asked for, into tensors that are passed in."""
    _say("parts")
    x, w, b, dout = _inputs(200, 72, 136, True, 5)
    xd, wd, bd, gd = _dev(x), [_dev(t) for t in w], [_dev(t) for t in b], _dev(dout)
    _, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
    want = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True)
    got = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, weight_grads=False)
    assert torch.equal(got[0], want[0]) and got[1:] == (None,) * 6
    for i in range(1, 7):
        held = torch.full_like(want[i], float("nan"))
        got = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, weight_grads=False, **{GRADS[i]: held})
        assert got[i] is held and torch.equal(held, want[i]) and sum(t is not None for t in got) == 2


def test_gradient_against_differences(V):
    """dx and the weights' gradients along directions against the difference of
    the loss in float64: off by the bars of the gradients and the step squared."""
    _say("differences")
    x, w, b, dout = _inputs(20, 40, 72, True, 21)
    wide = [_wide(t) for t in (x, *w, *b)]
    gw = _wide(dout)
    g = np.random.default_rng(22)
    ways = [g.standard_normal(t.shape) * np.abs(t).mean() for t in wide]
    loss = lambda s: float((tower.gated_mlp(*[t + s * v for t, v in zip(wide, ways)])["out"] * gw).sum())
    step = 1e-4
    slope = (loss(step) - loss(-step)) / (2 * step)
    dev = [_dev(t) for t in (x, *w, *b)]
    _, gate_up, hidden = V.gated_mlp(*dev, return_saved=True)
    got = V.gated_mlp_backward(_dev(dout), *dev[:4], gate_up, hidden, bias_grads=True)
    bars = _bars(wide[0], wide[1:4], wide[4:], gw, tower.gated_mlp(*wide, gw))
    ours = sum(float((_wide(t) * v).sum()) for t, v in zip(got, ways))
    bar = sum(float((bars[n] * np.abs(v)).sum()) for n, v in zip(GRADS, ways))
    assert abs(ours - slope) <= 1.05 * bar + 1e-6 * abs(slope)
    # each part of it is seen: without one of them the difference would show in its size
    assert all(float((np.abs(_wide(t)) * np.abs(v)).sum()) > 0 for t, v in zip(got, ways))


def test_empty(V):
    _say("empty")
    x, w, b, _ = _inputs(1, 72, 136, True, 5)
    xd, wd, bd = _dev(x)[:0], [_dev(t) for t in w], [_dev(t) for t in b]
    out, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
    assert out.shape == (0, 72) and gate_up.shape == (2, 0, 192) and hidden.shape == (0, 192)
    got = V.gated_mlp_backward(xd, xd, *wd, gate_up, hidden, bias_grads=True)
    assert got[0].shape == (0, 72) and all((t == 0).all() for t in got[1:])


def test_streams_graphs_and_workspaces(V):
    _say("streams and graphs")
    shape = (300, 264, 520)
    def make(seed):
        x, w, b, dout = _inputs(*shape, True, seed)
        return [_dev(t) for t in (x, *w, *b, dout)]

    def step(x, wg, wu, wd, bg, bu, bd, dout, **kw):
        out, gate_up, hidden = V.gated_mlp(x, wg, wu, wd, bg, bu, bd, return_saved=True, **kw)
        return (out, *V.gated_mlp_backward(dout, x, wg, wu, wd, gate_up, hidden, bias_grads=True, **kw))

    st = make(20)
    want = step(*st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(*st, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held = []
    for seed in (21, 22):
        st = make(seed)
        step(*st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*st)
        held.append((graph, st, outs))
    for turn in range(3):
        for i, (graph, st, outs) in enumerate(held):
            for t, new in zip(st, make(30 + 2 * turn + i)):
                t.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, step(*st)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("rows,d,h", [(1, 72, 136), (16, 72, 136), (17, 1280, 2048), (200, 1280, 640), (1500, 264, 4096), (2600, 640, 640),
                                      (4099, 72, 264), (20000, 128, 200)])
def test_the_same_bits_again(V, rows, d, h):
    """Few rows, split sums and whole tiles, from the same inputs next to other
    work on the card: bit for bit the same."""
    _say("again", (rows, d, h))
    x, w, b, dout = _inputs(rows, d, h, True, 9)
    xd, wd, bd, gd = _dev(x), [_dev(t) for t in w], [_dev(t) for t in b], _dev(dout)

    def step():
        out, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
        return (out, gate_up, hidden, *V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = [V.gated_mlp(xd, *wd, *bd) for _ in range(3)]
    got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got)) and all(torch.equal(o, want[0]) for o in other)


def test_past_32_bits(V):
    """A million rows of 2304 hidden values: rows of a large call against the
    float64 form, and the sums over all rows against sums in float64."""
    _say("a million rows")
    rows, d, h = 1_000_003, 64, 2304
    assert rows * h > 1 << 31
    x, w, b, _ = _inputs(64, d, h, True, 31)
    wd, bd = [_dev(t) for t in w], [_dev(t) for t in b]
    g = torch.Generator(device="cuda").manual_seed(32)
    x, dout = (torch.randn((rows, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, gate_up, hidden = V.gated_mlp(x, *wd, *bd, return_saved=True)
    got = V.gated_mlp_backward(dout, x, *wd, gate_up, hidden, bias_grads=True)
    for first in (0, rows // 2, rows - 64):
        at = slice(first, first + 64)
        wide = _wide(x[at]), [_wide(t) for t in w], [_wide(t) for t in b], _wide(dout[at])
        r = tower.gated_mlp(wide[0], *wide[1], *wide[2], wide[3])
        bars = _bars(*wide, r)
        _within(out[at], r["out"], bars["out"], "out")
        _within(got[0][at], r["dx"], bars["dx"], "dx")
        _within(gate_up[1, at], r["up"], bars["up"] + EPS * np.abs(r["up"]), "up")
    # the sums over all rows, from their operands as the kernels hold them: h and g, u as saved
    db, mag_b = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2))
    dw, mag = (torch.zeros((d, h), dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, rows, 1 << 16):
        dd, hh = dout[i:i + (1 << 16)].double(), hidden[i:i + (1 << 16)].double()
        db += dd.sum(0)
        mag_b += dd.abs().sum(0)
        dw += dd.T @ hh
        mag += dd.abs().T @ hh.abs()
    # additions on a value's way: over the rows of one of 128 x 8 row groups (or of a split), over those, and over a product's 16
    depth = rows / 1024 + 200
    assert ((got[6].double() - db).abs() <= depth * EPS * mag_b + EPS * db.abs()).all()
    assert ((got[3].double() - dw).abs() <= (rows + 8) * EPS * mag + U8 * dw.abs()).all()
    # a part of 64 rows left out, or taken twice, would show
    part = (dout[:64].double().T @ hidden[:64].double()).abs()
    assert (U8 * dw.abs()).median() < part.median()


def test_refusals(V):
    _say("refusals")
    x, w, b, dout = _inputs(4, 64, 72, True, 5)
    xd, (wg, wu, wd), bd, gd = _dev(x), [_dev(t) for t in w], [_dev(t) for t in b], _dev(dout)
    _, gate_up, hidden = V.gated_mlp(xd, wg, wu, wd, return_saved=True)
    small = torch.zeros(8, dtype=torch.uint8, device="cuda")
    for bad in (lambda: V.gated_mlp(xd.float(), wg, wu, wd), lambda: V.gated_mlp(xd, wg[:, :32], wu, wd), lambda: V.gated_mlp(xd, wg, wu[:64], wd),
                lambda: V.gated_mlp(xd, wg, wu, wd.t()), lambda: V.gated_mlp(xd, wg, wu, wd.t().contiguous()), lambda: V.gated_mlp(xd, wg.cpu(), wu, wd),
                lambda: V.gated_mlp(xd[0], wg, wu, wd), lambda: V.gated_mlp(xd, wg, wu, wd, bd[0][:8]),
                lambda: V.gated_mlp(xd, wg, wu, wd, bd[0].to(torch.bfloat16)), lambda: V.gated_mlp(xd, wg, wu, wd, out=xd),
                lambda: V.gated_mlp(xd, wg, wu, wd, out=xd[:2]), lambda: V.gated_mlp(xd, wg, wu, wd, workspace=small),
                lambda: V.gated_mlp(xd, wg, wu, wd, hidden=hidden), lambda: V.gated_mlp(xd, wg, wu, wd, return_saved=True, hidden=hidden[:, :72]),
                lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, None, hidden), lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, gate_up, None),
                lambda: V.gated_mlp_backward(gd[:2], xd, wg, wu, wd, gate_up, hidden),
                lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, gate_up[0], hidden),
                lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, gate_up, hidden, dx=gd),
                lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, gate_up, hidden, dw_up=wu),
                lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, gate_up, hidden, db_gate=bd[0], db_up=bd[0]),
                lambda: V.gated_mlp_backward(gd, xd, wg, wu, wd, gate_up, hidden, workspace=small)):
        with pytest.raises(V.MimoError):
            bad()


@pytest.mark.parametrize("rows,d,h", [(1, 64, 200), (37, 64, 200), (63, 71, 203), (1100, 1280, 1288), (14300, 944, 968)])
def test_infinities_of_the_weights(V, rows, d, h):
    """An infinite weight of the product back makes a hidden channel's dh
    infinite in every row: dg and du are too, all of one sign here, and so are
    the biases' gradients; the rows behind the last one, which are none, add no
    zero times infinity to them."""
    _say("infinite weights", (rows, d, h))
    x, w, b, dout = _inputs(rows, d, h, True, 17)
    xd, gd, wd, bd = _dev(x), _dev(dout), [_dev(t) for t in w], [_dev(t) for t in b]
    wd[2][3, 8], wd[2][5, h - 1] = float("inf"), float("-inf")
    _, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
    g, u = (gate_up[i, :, :h].double() for i in (0, 1))
    s = torch.sigmoid(g)
    one = torch.ones(rows, dtype=torch.bfloat16, device="cuda")
    gd[:, 3] = torch.copysign(one, (u * s * (1 + g * (1 - s)))[:, 8].float())
    gd[:, 5] = torch.copysign(one, (g * s)[:, h - 1].float())
    got = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True)
    db_gate, db_up = got[4], got[5]
    assert db_gate[8] == float("inf") and db_up[h - 1] == float("-inf")
    keep = torch.ones(h, dtype=torch.bool, device="cuda")
    keep[[8, h - 1]] = False
    assert torch.isfinite(db_gate[keep]).all() and torch.isfinite(db_up[keep]).all()
    with np.errstate(invalid="ignore"):
        r = tower.gated_mlp(_wide(xd), *[_wide(t) for t in wd], *[_wide(t) for t in bd], _wide(gd))
    for name, t in (("db_gate", db_gate), ("db_up", db_up)):
        want = torch.from_numpy(r[name]).cuda()
        assert torch.equal(torch.isinf(t), torch.isinf(want)) and torch.equal(torch.isnan(t), torch.isnan(want)), name


@pytest.mark.parametrize("rows,d,h", mlp_tiles.SIZES)
def test_whole_tiles_next_to_parts(V, rows, d, h):
    """Launches of whole tiles and, behind them, tiles in parts of K: of one
    product, and of the three weights' gradients, at each tile size."""
    _check(V, rows, d, h, True, 13)


def test_each_gradient_against_differences(V):
    """Each tensor's gradient along the signs of the oracle's, against the
    central difference of the loss in float64: off by that gradient's own bars,
    and by the step squared times the loss's third derivative (relative to the
    first, the square of what a step of one moves g by, some 50: 3e-7 at most for
    a step of 1e-4 and a direction of the tensor's size).  The bar is far below
    the slope, so a gradient that is missing, halved or of the wrong sign shows."""
    _say("differences, one by one")
    x, w, b, dout = _inputs(20, 40, 72, True, 21)
    wide = [_wide(t) for t in (x, *w, *b)]
    gw = _wide(dout)
    dev = [_dev(t) for t in (x, *w, *b)]
    _, gate_up, hidden = V.gated_mlp(*dev, return_saved=True)
    got = V.gated_mlp_backward(_dev(dout), *dev[:4], gate_up, hidden, bias_grads=True)
    r = tower.gated_mlp(*wide, gw)
    bars = _bars(wide[0], wide[1:4], wide[4:], gw, r)
    step = 1e-4
    for i, name in enumerate(GRADS):
        way = np.sign(r[name]) * np.abs(wide[i]).mean()
        loss = lambda s: float((tower.gated_mlp(*wide[:i], wide[i] + s * way, *wide[i + 1:])["out"] * gw).sum())
        slope = (loss(step) - loss(-step)) / (2 * step)
        bar = 1.05 * float((bars[name] * np.abs(way)).sum()) + 1e-6 * abs(slope)
        assert abs(float((_wide(got[i]) * way).sum()) - slope) <= bar and bar < slope / 4, name


def test_without_the_inputs_gradient(V):
    """dx left out: the other gradients' bits are the same, on another stream
    too; made all the same where it is passed in."""
    _say("without dx")
    x, w, b, dout = _inputs(200, 72, 136, True, 5)
    xd, wd, bd, gd = _dev(x), [_dev(t) for t in w], [_dev(t) for t in b], _dev(dout)
    _, gate_up, hidden = V.gated_mlp(xd, *wd, *bd, return_saved=True)
    want = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in ({}, {"stream": side}):
        got = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, bias_grads=True, input_grad=False, **kw)
        side.synchronize()
        assert got[0] is None and all(torch.equal(a, c) for a, c in zip(got[1:], want[1:]))
    held = torch.full_like(xd, float("nan"))
    got = V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, dx=held, weight_grads=False, input_grad=False)
    assert got[0] is held and torch.equal(held, want[0]) and got[1:] == (None,) * 6
    assert V.gated_mlp_backward(gd, xd, *wd, gate_up, hidden, weight_grads=False, input_grad=False) == (None,) * 7
