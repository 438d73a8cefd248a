"""GPU parity of chunked attention, forward and backward, against the float64
form on the same bf16 inputs.

Bars, derived from the arithmetic (u = 2^-8, bf16's largest relative rounding;
e = 2^-24, float32's).  With S = max_j scale sum |q||k| + |sink| of a row and
n keys seen, a logit is off by at most (D + 4) e S, and a probability, with
its exponent, sum and rescaling, by the relative
  E = 2 (D + 4) e S + (n + 16) 2 e.
  out:  u sum p|v| (p as a bf16 operand) + E sum p|v| + u |out|
  lse:  E + 4 e |lse|
  dp:   (D + 2) e sum |do||v|;   delta: sum |do| (bar of out) + (D + 2) e sum |do||out|
  ds:   p (|dp - delta| E + bar of dp + bar of delta), plus u of the result as an operand
  dq:   scale sum_j (bar of ds) |k| + n e scale sum |ds||k| + u |dq|; dk, dv alike over rows and heads
  dsink: uses sum_j p dp in place of delta, so no bf16 rounding enters:
        sum_i p_i0 (|dp - delta| E + bar of dp + sum_j p (|dp| E + bar of dp + n e |dp|)) + rows e sum |ds_i0|
A second-order term of each product of two small numbers is covered by a
factor of 1.01.
"""
import numpy as np
import pytest

from oracle import tower

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U, EPS = 2.0 ** -8, 2.0 ** -24
SLACK = 1.01


def _say(*a):
    print("[gpu-attention]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _inputs(rows, hq, hk, d, seed, sink, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    draw = lambda h: (torch.randn((rows, h, d), generator=g) * spread).to(torch.bfloat16)
    q, k, v, do = draw(hq), draw(hk), draw(hk), draw(hq)
    s = torch.randn(hq, generator=g) * 2 if sink else None
    return q, k, v, do, s


def _wide(t):
    return None if t is None else t.double().numpy()


def _within(got, want, bar, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    bad = err > SLACK * bar + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float((err / (bar + 1e-30)).max()))


def _forward_bars(r, d):
    rel = 2 * (d + 4) * EPS * r["abs_s"] + (r["seen"] + 16) * 2 * EPS  # [hq, rows]
    e = rel.T[:, :, None]
    return rel, (U + e) * r["abs_out"] + U * np.abs(r["out"]), rel + 4 * EPS * np.abs(np.where(np.isinf(r["lse"]), 0, r["lse"]))


def _backward_bars(q, k, v, do, r, scale, rel, out_bar, d):
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dsink, abs0 = np.zeros(q.shape[1]), np.zeros(q.shape[1])
    terms = np.zeros(k.shape[:2])  # summands of each key's gradients
    for a, b, h, g, p, dp, ds in r["parts"]:
        n = b - a
        e = rel[h, a:b][:, None]
        ado, ak, aq = np.abs(do[a:b, h]), np.abs(k[a:b, g]), np.abs(q[a:b, h])
        dp_bar = (d + 2) * EPS * (ado @ np.abs(v[a:b, g]).T)
        delta_bar = ((ado * out_bar[a:b, h]).sum(1) + (d + 2) * EPS * (ado * np.abs(r["out"][a:b, h])).sum(1))[:, None]
        away = np.where(p > 0, np.abs(ds) / np.where(p > 0, p, 1), 0)
        ds_bar = p * (away * e + dp_bar + delta_bar)
        ds_bar += U * (np.abs(ds) + ds_bar)
        dq[a:b, h] += scale * (ds_bar + n * EPS * np.abs(ds)) @ ak
        dk[a:b, g] += scale * ds_bar.T @ aq
        dv[a:b, g] += ((U + e) * p).T @ ado
        terms[a:b, g] += n
        mean_bar = (p * (np.abs(dp) * e + dp_bar + n * EPS * np.abs(dp))).sum(1)
        dsink[h] += (p[:, 0] * (away[:, 0] * e[:, 0] + dp_bar[:, 0] + mean_bar)).sum()
        abs0[h] += np.abs(ds[:, 0]).sum()
    for a, b, h, g, p, dp, ds in r["parts"]:
        many = terms[a:b, g][:, None] * EPS
        dk[a:b, g] += many * scale * (np.abs(ds).T @ np.abs(q[a:b, h]))
        dv[a:b, g] += many * (p.T @ np.abs(do[a:b, h]))
    dsink += q.shape[0] * EPS * abs0 + EPS * np.abs(r["dsink"])
    return dq + U * np.abs(r["dq"]), dk + U * np.abs(r["dk"]), dv + U * np.abs(r["dv"]), dsink


def _check(V, lengths, hq, hk, d, window, sink, seed, tail=0, scale=None, spread=1.0):
    _say(lengths, (hq, hk, d), "window", window, "sink", sink)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    rows = int(cu[-1]) + tail
    q, k, v, do, s = _inputs(rows, hq, hk, d, seed, sink, spread)
    scale_used = d ** -0.5 if scale is None else scale
    r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), cu, window, scale, _wide(s), _wide(do))
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (q, k, v, do)]
    sd = None if s is None else s.cuda()
    before = V.dispatch_count()
    out, lse = V.chunk_attention(*dev[:3], cud, window=window, scale=scale, sink=sd, return_lse=True)
    grads = V.chunk_attention_backward(dev[3], *dev[:3], out, lse, cud, window=window, scale=scale, sink=sd)
    torch.cuda.synchronize()
    # forward, dq, dk and dv, and the join of dk's and dv's slices
    assert V.dispatch_count() - before in (3, 4)
    rel, out_bar, lse_bar = _forward_bars(r, d)
    end = int(cu[-1])
    _within(out[:end], r["out"][:end], out_bar[:end], "out")
    _within(lse[:, :end], r["lse"][:, :end], lse_bar[:, :end], "lse")
    bars = _backward_bars(_wide(q), _wide(k), _wide(v), _wide(do), r, scale_used, rel, out_bar, d)
    for got, name, bar in zip(grads, ("dq", "dk", "dv", "dsink"), bars):
        if name == "dsink":
            if sink:
                _within(got, r[name], bar, name)
            else:
                assert got is None
        else:
            _within(got[:end], r[name][:end], bar[:end], name)


@pytest.mark.parametrize("lengths", [[1], [2, 1, 3], [31, 32, 33], [63, 64, 65], [127, 128, 129], [0, 5, 0, 0, 200, 0], [516]])
@pytest.mark.parametrize("window,sink", [(-1, False), (-1, True), (64, True), (5, False), (0, True)])
def test_lengths(V, lengths, window, sink):
    _check(V, lengths, 4, 2, 64, window, sink, seed=sum(lengths) + window)


@pytest.mark.parametrize("lengths", [[1], [2, 1, 3], [31, 33], [64, 63], [0, 5, 0, 0, 129, 0], [300]])
@pytest.mark.parametrize("window,sink", [(-1, False), (64, True), (5, True), (0, True)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (4, 1, 88), (12, 3, 128)])
def test_lengths_of_four_heads(V, lengths, window, sink, hq, hk, d):
    """Heads in groups of four, which share a workgroup."""
    _check(V, lengths, hq, hk, d, window, sink, seed=sum(lengths) + window + hk)


@pytest.mark.parametrize("hq,hk,d,window", [(256, 256, 64, -1), (256, 256, 64, 20), (1024, 256, 64, -1), (256, 256, 128, 50)])
def test_sums_that_are_not_sliced(V, hq, hk, d, window):
    """Enough key heads that dk's and dv's sums are not split among workgroups."""
    _check(V, [70, 130], hq, hk, d, window, True, seed=hq + d)


@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (8, 8, 8), (8, 2, 32), (6, 1, 72), (8, 2, 80), (4, 2, 128), (4, 4, 96),
                                     (12, 4, 56), (32, 8, 64), (3, 3, 120)])
@pytest.mark.parametrize("window", [-1, 40])
def test_heads(V, hq, hk, d, window):
    _check(V, [75, 140], hq, hk, d, window, True, seed=hq * d)


def test_many_chunks(V):
    rng = np.random.default_rng(3)
    lengths = [int(n) for n in rng.integers(0, 12, 300)]
    _check(V, lengths, 2, 1, 64, -1, True, seed=11)
    _check(V, lengths, 2, 1, 64, 3, False, seed=12)


def test_long_chunk(V):
    _check(V, [2300], 2, 1, 64, -1, True, seed=13)
    _check(V, [2300], 1, 1, 128, 300, True, seed=14)
    _check(V, [2300], 32, 16, 64, -1, True, seed=22)
    _check(V, [1500, 700], 32, 32, 64, 64, True, seed=23)
    _check(V, [700, 900], 40, 10, 128, -1, False, seed=24)


@pytest.mark.parametrize("scale,spread", [(0.02, 1.0), (1.0, 2.0), (0.125, 6.0)])
def test_scales(V, scale, spread):
    """Flat and peaked softmaxes; logits up to some hundreds."""
    _check(V, [100, 300], 4, 2, 64, -1, True, seed=15, scale=scale, spread=spread)


@pytest.mark.parametrize("size", [1e4, 1e6, 1e8])
def test_large_logits(V, size):
    """Logits of up to 10^8: one key takes each row, whichever has the largest
    logit by more than float32's spacing there."""
    _say("large logits", size)
    n, d = 300, 64
    g = torch.Generator().manual_seed(33)
    k = torch.nn.functional.one_hot(torch.arange(n) % d, d).to(torch.bfloat16)[:, None]
    k[64:] *= 0.5  # shorter copies of the first 64
    q = (torch.nn.functional.one_hot(torch.randint(0, d, (n,), generator=g), d) * size).to(torch.bfloat16)[:, None]
    v = torch.randn((n, 1, d), generator=g).to(torch.bfloat16)
    r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), [0, n], -1, 1.0)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = V.chunk_attention(q.cuda(), k.cuda(), v.cuda(), cu, scale=1.0, return_lse=True)
    # one probability, rounded to bf16, over itself; lse by way of powers of
    # two: two constants, their products, the maximum, and the sum with its log
    _within(out, r["out"], 2 * U * np.abs(r["out"]), "out")
    _within(lse, r["lse"], 6 * EPS * np.abs(r["lse"]), "lse")


def test_rising_logits(V):
    """Every step's maximum outgrows the last one's: keys grow along the chunk."""
    _say("rising logits")
    n, d = 700, 64
    q, k, v, do, _ = _inputs(n, 1, 1, d, 16, False)
    q = q.abs()
    k = (k.abs() * torch.linspace(0, 4, n)[:, None, None]).to(torch.bfloat16)
    r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), [0, n], -1, None, None, _wide(do))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = V.chunk_attention(q.cuda(), k.cuda(), v.cuda(), cu, return_lse=True)
    grads = V.chunk_attention_backward(do.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, cu)
    rel, out_bar, lse_bar = _forward_bars(r, d)
    _within(out, r["out"], out_bar, "out")
    _within(lse, r["lse"], lse_bar, "lse")
    bars = _backward_bars(_wide(q), _wide(k), _wide(v), _wide(do), r, d ** -0.5, rel, out_bar, d)
    for got, name, bar in zip(grads[:3], ("dq", "dk", "dv"), bars):
        _within(got, r[name], bar, name)


def test_rows_that_see_nothing(V):
    """A sink of -inf takes key 0 away; where it was alone, nothing is left."""
    _say("rows that see nothing")
    lengths = [1, 4, 1, 70]
    cu_host = [0, 1, 5, 6, 76]
    q, k, v, do, _ = _inputs(76, 2, 1, 64, 17, False)
    sink = torch.tensor([-float("inf"), 0.5])
    cu = torch.tensor(cu_host, dtype=torch.int32, device="cuda")
    for window in (-1, 0, 2):
        r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), cu_host, window, None, _wide(sink), _wide(do))
        out, lse = V.chunk_attention(q.cuda(), k.cuda(), v.cuda(), cu, window=window, sink=sink.cuda(), return_lse=True)
        grads = V.chunk_attention_backward(do.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, cu, window=window,
                                           sink=sink.cuda())
        none = np.isneginf(r["lse"])
        assert none.any() and (torch.isneginf(lse).cpu().numpy() == none).all()
        assert (out.float().cpu().numpy().transpose(1, 0, 2)[none] == 0).all()
        rel, out_bar, _ = _forward_bars(r, 64)
        _within(out, r["out"], out_bar, "out")
        bars = _backward_bars(_wide(q), _wide(k), _wide(v), _wide(do), r, 0.125, rel, out_bar, 64)
        for got, name, bar in zip(grads, ("dq", "dk", "dv", "dsink"), bars):
            _within(got, r[name], bar, f"{name} window {window}")


def test_sinks_of_any_size(V):
    """Sinks that take a row for themselves, and sinks that vanish."""
    _say("sinks of any size")
    cu_host, n = [0, 70, 200], 200
    q, k, v, do, _ = _inputs(n, 6, 2, 64, 25, False)
    sink = torch.tensor([-200.0, -50.0, 30.0, 95.0, 130.0, 600.0])
    r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), cu_host, -1, None, _wide(sink), _wide(do))
    cu = torch.tensor(cu_host, dtype=torch.int32, device="cuda")
    out, lse = V.chunk_attention(q.cuda(), k.cuda(), v.cuda(), cu, sink=sink.cuda(), return_lse=True)
    grads = V.chunk_attention_backward(do.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, cu, sink=sink.cuda())
    rel, out_bar, lse_bar = _forward_bars(r, 64)
    _within(out, r["out"], out_bar, "out")
    _within(lse, r["lse"], lse_bar, "lse")
    bars = _backward_bars(_wide(q), _wide(k), _wide(v), _wide(do), r, 0.125, rel, out_bar, 64)
    for got, name, bar in zip(grads, ("dq", "dk", "dv", "dsink"), bars):
        _within(got, r[name], bar, name)


def test_sinks_that_are_not_finite_stay_with_key_0(V):
    """Rows whose band does not hold key 0 share its block, and have none of
    its sink, whatever it is."""
    _say("sinks that are not finite")
    cu_host, n, window = [0, 40, 140], 140, 5
    q, k, v, _, _ = _inputs(n, 4, 2, 64, 26, False)
    cu = torch.tensor(cu_host, dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (q, k, v)]
    sink = torch.tensor([float("inf"), float("nan"), -float("inf"), 2.0], device="cuda")
    out, lse = V.chunk_attention(*dev, cu, window=window, sink=sink, return_lse=True)
    plain, plain_lse = V.chunk_attention(*dev, cu, window=window, return_lse=True)
    r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), cu_host, window)
    _, out_bar, lse_bar = _forward_bars(r, 64)
    for a, b in zip(cu_host[:-1], cu_host[1:]):
        away = slice(a + window + 1, b)
        assert torch.equal(out[away], plain[away]) and torch.equal(lse[:, away], plain_lse[:, away])
        _within(out[away], r["out"][away], out_bar[away], "out")
        _within(lse[:, away], r["lse"][:, away], lse_bar[:, away], "lse")


@pytest.mark.parametrize("window", [-1, 0, 5])
def test_sinks_beyond_the_range(V, window):
    """The type's lowest and highest values and what lies before them: key 0
    has nothing, or all, as by the definition in 64 bits.  lse and the bars are
    those of the sink at the range's end, which is what it counts as."""
    _say("sinks beyond the range, window", window)
    big = float(torch.finfo(torch.float32).max)
    cu_host, n = [0, 1, 71, 111], 111
    sink = torch.tensor([-big, -1e30, -1e9, -1e5, 1e5, 1e9, big, float("inf")])
    q, k, v, do, _ = _inputs(n, 8, 2, 64, 27, False)
    wide = [_wide(t) for t in (q, k, v)]
    by_definition = tower.chunk_attention(*wide, cu_host, window, None, _wide(sink.clamp(-big, big)), _wide(do))
    r = tower.chunk_attention(*wide, cu_host, window, None, _wide(sink.clamp(-8192, 8192)), _wide(do))
    for name in ("out", "dq", "dk", "dv", "dsink"):
        np.testing.assert_allclose(r[name], by_definition[name], rtol=1e-9, atol=1e-9)
    cu = torch.tensor(cu_host, dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = V.chunk_attention(*dev, cu, window=window, sink=sink.cuda(), return_lse=True)
    grads = V.chunk_attention_backward(do.cuda(), *dev, out, lse, cu, window=window, sink=sink.cuda())
    rel, out_bar, lse_bar = _forward_bars(r, 64)
    _within(out, by_definition["out"], out_bar, "out")
    _within(lse, r["lse"], lse_bar, "lse")
    bars = _backward_bars(_wide(q), _wide(k), _wide(v), _wide(do), r, 0.125, rel, out_bar, 64)
    for got, name, bar in zip(grads, ("dq", "dk", "dv", "dsink"), bars):
        _within(got, by_definition[name], bar, f"{name} window {window}")
    clamped = V.chunk_attention(*dev, cu, window=window, sink=sink.clamp(-8192, 8192).cuda(), return_lse=True)
    assert torch.equal(out, clamped[0]) and torch.equal(lse, clamped[1])


def test_strides_and_slices(V):
    """Slices of one packed projection, head-major tensors, a shared key head
    by a stride of zero, and gradients into slices: the same bits as dense ones."""
    _say("strides")
    n, hq, hk, d = 150, 4, 2, 64
    q, k, v, do, s = (None if t is None else t.cuda() for t in _inputs(n, hq, hk, d, 18, True))
    cu = torch.tensor([0, 40, 150], dtype=torch.int32, device="cuda")
    out, lse = V.chunk_attention(q, k, v, cu, window=30, sink=s, return_lse=True)
    want = V.chunk_attention_backward(do, q, k, v, out, lse, cu, window=30, sink=s)

    packed = torch.zeros((n, hq + 2 * hk, d), dtype=torch.bfloat16, device="cuda")
    pq, pk, pv = packed[:, :hq], packed[:, hq:hq + hk], packed[:, hq + hk:]
    pq.copy_(q), pk.copy_(k), pv.copy_(v)
    major = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    for qq, kk, vv, dd in ((pq, pk, pv, do), (major(q), major(k), major(v), major(do))):
        o = torch.empty((hq, n, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        o2, l2 = V.chunk_attention(qq, kk, vv, cu, window=30, sink=s, out=o, return_lse=True)
        assert o2 is o and torch.equal(o, out) and torch.equal(l2, lse)
        grads = torch.full((n, hq + 2 * hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
        got = V.chunk_attention_backward(dd, qq, kk, vv, o, l2, cu, window=30, sink=s, dq=grads[:, :hq],
                                         dk=grads[:, hq:hq + hk], dv=grads[:, hq + hk:])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    one = k[:, :1].expand(n, hk, d)
    assert one.stride(1) == 0
    a = V.chunk_attention(q, one, v, cu)
    b = V.chunk_attention(q, one.contiguous(), v, cu)
    assert torch.equal(a, b)


def test_rows_behind_the_last_chunk(V):
    """Neither read nor written, in any tensor; nor is what is around slices."""
    _say("rows behind the last chunk")
    n, tail, hq, hk, d = 90, 37, 4, 2, 64
    q, k, v, do, s = _inputs(n + tail, hq, hk, d, 19, True)
    for t in (q, k, v, do):
        t[n:] = float("nan")
    cu = torch.tensor([0, 50, 90], dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (q, k, v, do)]
    s = s.cuda()
    out = torch.full((n + tail, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, n + tail), 3.0, device="cuda")
    V.chunk_attention(*dev[:3], cu, sink=s, out=out, lse=lse)
    grads = [torch.full_like(t, 3.0) for t in dev[:3]]
    _, _, _, dsink = V.chunk_attention_backward(dev[3], *dev[:3], out, lse, cu, sink=s, dq=grads[0], dk=grads[1],
                                                dv=grads[2])
    for t in (out, *grads):
        assert (t[n:] == 3).all() and torch.isfinite(t).all()
    assert (lse[:, n:] == 3).all() and torch.isfinite(lse).all()
    short = [t[:n].contiguous() for t in dev]
    o, l = V.chunk_attention(*short[:3], cu, sink=s, return_lse=True)
    want = V.chunk_attention_backward(short[3], *short[:3], o, l, cu, sink=s)
    assert torch.equal(o, out[:n]) and torch.equal(l, lse[:, :n]) and torch.equal(dsink, want[3])
    for a, b in zip(grads, want):
        assert torch.equal(a[:n], b)


@pytest.mark.parametrize("hq,hk", [(8, 2), (2, 2)])
@pytest.mark.parametrize("window", [-1, 40])
@pytest.mark.parametrize("first", [31, 32, 200, 1000])
def test_rows_in_front_of_the_first_chunk(V, hq, hk, window, first):
    """Boundaries that do not start at 0, by more than a tile: the rows in
    front are neither read nor written, and the others have the values of a
    call without them."""
    _say("rows in front", (hq, hk), window, first)
    n, d = 330, 64
    rng = np.random.default_rng(first)
    for lengths in ([130, 0, 200], [int(x) for x in rng.multinomial(n, [1 / 90] * 90)]):
        q, k, v, do, s = (t.cuda() for t in _inputs(first + n, hq, hk, d, 29, True))
        for t in (q, k, v, do):
            t[:first] = float("nan")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 3.0), torch.full((hq, first + n), 3.0, device="cuda")
        V.chunk_attention(q, k, v, cu + first, window=window, sink=s, out=out, lse=lse)
        grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
        _, _, _, dsink = V.chunk_attention_backward(do, q, k, v, out, lse, cu + first, window=window, sink=s, dq=grads[0],
                                                    dk=grads[1], dv=grads[2])
        for t in (out, *grads):
            assert (t[:first] == 3).all()
        assert (lse[:, :first] == 3).all()
        x = [t[first:].double().cpu().numpy() for t in (q, k, v, do)]
        r = tower.chunk_attention(*x[:3], cu.cpu().numpy(), window, None, _wide(s.cpu()), x[3])
        rel, out_bar, lse_bar = _forward_bars(r, d)
        _within(out[first:], r["out"], out_bar, "out")
        _within(lse[:, first:], r["lse"], lse_bar, "lse")
        bars = _backward_bars(*x, r, d ** -0.5, rel, out_bar, d)
        for got, name, bar in zip([g[first:] for g in grads] + [dsink], ("dq", "dk", "dv", "dsink"), bars):
            _within(got, r[name], bar, name)


def test_other_chunks_are_not_touched(V):
    """What is not finite in one chunk reaches no other."""
    _say("chunks apart")
    q, k, v, do, _ = (None if t is None else t.cuda() for t in _inputs(200, 2, 2, 64, 20, False))
    cu = torch.tensor([0, 70, 131, 200], dtype=torch.int32, device="cuda")
    a, la = V.chunk_attention(q, k, v, cu, return_lse=True)
    want = V.chunk_attention_backward(do, q, k, v, a, la, cu)
    for t in (q, k, v, do):
        t[70:131] = float("inf")
        t[80:90] = float("nan")
    b, lb = V.chunk_attention(q, k, v, cu, return_lse=True)
    got = V.chunk_attention_backward(do, q, k, v, b, lb, cu)
    for rows in (slice(0, 70), slice(131, 200)):
        assert torch.equal(a[rows], b[rows]) and torch.equal(la[:, rows], lb[:, rows])
        for x, y in zip(got[:3], want[:3]):
            assert torch.equal(x[rows], y[rows])


def test_bad_boundaries_stay_inside(V):
    """A boundary outside the rows, or a descending pair, makes its chunk empty."""
    _say("bad boundaries")
    q, k, v, do, _ = (None if t is None else t.cuda() for t in _inputs(64, 1, 1, 64, 21, False))
    good = torch.tensor([0, 20, 20, 20], dtype=torch.int32, device="cuda")
    want = V.chunk_attention(q, k, v, good)
    for bad in ([0, 20, 65, 2 ** 31 - 1], [0, 20, -5, 20], [0, 20, 10, -(2 ** 31)]):
        out = torch.full_like(q, 3.0)
        V.chunk_attention(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        assert torch.equal(out[:10], want[:10])


@pytest.mark.parametrize("hq,hk", [(8, 2), (2, 2)])
@pytest.mark.parametrize("window", [-1, 40])
def test_boundaries_that_do_not_ascend(V, hq, hk, window):
    """Chunks of several tiles, in any order, one over the other, or outside the
    rows: nothing around the outputs and the workspace is written, and the next
    call is right."""
    _say("boundaries that do not ascend", (hq, hk), window)
    n, d, guard = 600, 64, 3
    q, k, v, do, s = (t.cuda() for t in _inputs(n, hq, hk, d, 28, True))
    good = torch.tensor([0, 130, 130, 600], dtype=torch.int32, device="cuda")
    want, lse = V.chunk_attention(q, k, v, good, window=window, sink=s, return_lse=True)
    want = (want, lse, *V.chunk_attention_backward(do, q, k, v, want, lse, good, window=window, sink=s))

    def guarded(shape, dtype, edge):
        """A tensor of zeros in the middle of one that holds sevens."""
        t = torch.full((edge * 2 + int(np.prod(shape)),), 7, dtype=dtype, device="cuda")
        t[edge:-edge] = 0
        return t, t[edge:-edge].view(shape)

    for bad in ([500, 600, 0, 400], [0, 700, 300, 600], [-3, 200, 100, 2 ** 31 - 1, 0, 600], [600, 400, 200, 0],
                [0, 600, 0, 600], [-(2 ** 31), 2 ** 31 - 1, -(2 ** 31)]):
        _say(bad)
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        held = [guarded(shape, dtype, edge) for shape, dtype, edge in (
            ((n, hq, d), torch.bfloat16, guard * hq * d), ((hq, n), torch.float32, 64), ((n, hq, d), torch.bfloat16, guard * hq * d),
            ((n, hk, d), torch.bfloat16, guard * hk * d), ((n, hk, d), torch.bfloat16, guard * hk * d), ((hq,), torch.float32, 64),
            ((V.chunk_attention_workspace_bytes(n, hq, hk, d, len(bad) - 1),), torch.uint8, 4096))]
        out, l, dq, dk, dv, dsink, workspace = (inner for _, inner in held)
        V.chunk_attention(q, k, v, cu, window=window, sink=s, out=out, lse=l)
        V.chunk_attention_backward(do, q, k, v, out, l, cu, window=window, sink=s, dq=dq, dk=dk, dv=dv, dsink=dsink,
                                   workspace=workspace)
        torch.cuda.synchronize()
        for whole, inner in held:
            edge = (whole.numel() - inner.numel()) // 2
            assert (whole[:edge] == 7).all() and (whole[-edge:] == 7).all()
    again, lse = V.chunk_attention(q, k, v, good, window=window, sink=s, return_lse=True)
    again = (again, lse, *V.chunk_attention_backward(do, q, k, v, again, lse, good, window=window, sink=s))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_streams_and_graphs(V):
    """A stream of the caller's, and two captured calls that are replayed
    between eager ones with new inputs and boundaries, each with a workspace of
    its own: every replay gives the eager bits."""
    _say("streams and graphs")
    hq, hk, d, n = 4, 2, 64, 300
    mk = lambda seed: [None if t is None else t.cuda() for t in _inputs(n, hq, hk, d, seed, True)]
    cus = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, 100, 300], [0, 299, 300], [0, 0, 200])]

    def eager(x, cu):
        o, l = V.chunk_attention(*x[:3], cu, window=50, sink=x[4], return_lse=True)
        return (o, *V.chunk_attention_backward(x[3], *x[:3], o, l, cu, window=50, sink=x[4]))

    x = mk(30)
    want = eager(x, cus[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l = V.chunk_attention(*x[:3], cus[0], window=50, sink=x[4], return_lse=True, stream=side)
    got = (o, *V.chunk_attention_backward(x[3], *x[:3], o, l, cus[0], window=50, sink=x[4], stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    held = []
    for seed in (31, 32):
        st = [t.clone() for t in mk(seed)]
        cu = cus[0].clone()
        eager(st, cu)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = eager(st, cu)
        held.append((graph, st, cu, outs))
    for turn in range(3):
        for i, (graph, st, cu, outs) in enumerate(held):
            for t, new in zip(st, mk(40 + 2 * turn + i)):
                t.copy_(new)
            cu.copy_(cus[(turn + i) % 3])
            end = int(cu[-1])
            graph.replay()
            torch.cuda.synchronize()
            want = eager(st, cu)
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                a, b = (a, b) if a.dim() == 1 else (a[:end], b[:end])
                assert torch.equal(a, b)


def test_empty(V):
    _say("empty")
    z = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = V.chunk_attention(z, z, z, cu, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    sink = torch.ones(4, device="cuda")
    dq, dk, dv, dsink = V.chunk_attention_backward(z, z, z, z, out, lse, cu, sink=sink)
    assert dq.shape == z.shape and (dsink == 0).all()
    x = torch.ones((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(x, 2.0)
    V.chunk_attention(x, x, x, torch.zeros(3, dtype=torch.int32, device="cuda"), out=o)
    assert (o == 2).all()
