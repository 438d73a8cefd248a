"""The tower's operators together, as a block uses them, over a plan's rows:
pixel rows -> 8-bit embedding -> layer norm -> 8-bit projection to q, k and v
(one output, sliced) -> attention over the plan's chunks, with a band and
sinks; and back again, the gradients of q, k and v written into slices of one
tensor, through the projection (a plain product) to the norm's.

Every stage is held to the float64 form on the values that it was given, with
the bars of its own tests.  And sizes past 2^31 values, where a part of a
large call has to equal the same part called alone.
"""
import numpy as np
import pytest

import test_gpu_attention as A
import test_gpu_norm as N
import workloads as W
from oracle import tower

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _say(*a):
    print("[gpu-tower]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _wide(t):
    return t.double().cpu().numpy()


def _linear_bar(ref, mag, out):
    u = 2.0 ** -8 if out.dtype == torch.bfloat16 else A.EPS
    return 3.01 * A.EPS * mag + A.EPS * (np.abs(ref) + mag) + u * np.abs(ref)


@pytest.mark.parametrize("window", [-1, 16])
def test_block_over_a_plan(V, window):
    _say("block, window", window)
    b = W.media_batch([(1, 200, 300, 3), (5, 64, 96, 3), (1, 45, 77, 4), (1, 1, 64, 3)], seed=81)
    plan = V.plan_media(b.items)
    src = V.processor.upload_sources(b.packed, plan)
    rows = V.preprocess(src, plan, mean=b.mean, std=b.std, out_dtype="bf16")["pixel_values"]
    cu = V.vit_tables(plan)["cu_seqlens"].cuda()
    cu_host = cu.cpu().numpy()
    n, e, hq, hk, d = plan.total_rows, 512, 8, 2, 64
    g = torch.Generator().manual_seed(82)
    draw = lambda *s: torch.randn(s, generator=g)
    wq, ws = V.quantize_rows((draw(e, 1536) * 0.02).cuda())
    pw = draw((hq + 2 * hk) * d, e) * 0.05
    pq, ps = V.quantize_rows(pw.cuda())
    weight, bias, sink = (1 + 0.2 * draw(e)).cuda(), (0.2 * draw(e)).cuda(), draw(hq).cuda()

    xq, xs = V.quantize_rows(rows)
    emb = V.quantized_linear(xq, xs, wq, ws, None, out_dtype="f32")
    ref, mag = tower.quantized_linear(xq.cpu().numpy(), xs.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy())
    assert (np.abs(_wide(emb) - ref) <= 1.01 * _linear_bar(ref, mag, emb)).all()
    want_q, want_s = tower.quantize_rows(rows.float().cpu().numpy())
    assert np.array_equal(xq.cpu().numpy(), want_q) and np.array_equal(xs.cpu().numpy(), want_s)

    normed, mean, rstd = V.layer_norm(emb, weight, bias, out_dtype="bf16", return_stats=True)
    r = tower.layer_norm(_wide(emb), _wide(weight), _wide(bias), N.NORM_EPS)
    _, _, out_bar = N._bars(_wide(emb), None, _wide(weight), _wide(bias), r)
    N._within(normed, r["out"], out_bar + N.ROUND[torch.bfloat16] * np.abs(r["out"]), "norm")

    nq, ns = V.quantize_rows(normed)
    qkv = V.quantized_linear(nq, ns, pq, ps).view(n, hq + 2 * hk, d)
    ref, mag = tower.quantized_linear(nq.cpu().numpy(), ns.cpu().numpy(), pq.cpu().numpy(), ps.cpu().numpy())
    assert (np.abs(_wide(qkv).reshape(n, -1) - ref) <= 1.01 * _linear_bar(ref, mag, qkv)).all()

    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    out, lse = V.chunk_attention(q, k, v, cu, window=window, sink=sink, return_lse=True)
    dout = draw(n, hq, d).to(torch.bfloat16).cuda()
    r = tower.chunk_attention(_wide(q), _wide(k), _wide(v), cu_host, window, None, _wide(sink), _wide(dout))
    rel, out_bar, lse_bar = A._forward_bars(r, d)
    A._within(out, r["out"], out_bar, "out")
    A._within(lse, r["lse"], lse_bar, "lse")

    dqkv = torch.empty_like(qkv)
    _, _, _, dsink = V.chunk_attention_backward(dout, q, k, v, out, lse, cu, window=window, sink=sink, dq=dqkv[:, :hq],
                                                dk=dqkv[:, hq:hq + hk], dv=dqkv[:, hq + hk:])
    bars = A._backward_bars(_wide(q), _wide(k), _wide(v), _wide(dout), r, d ** -0.5, rel, out_bar, d)
    for got, name, bar in zip((dqkv[:, :hq], dqkv[:, hq:hq + hk], dqkv[:, hq + hk:], dsink), ("dq", "dk", "dv", "dsink"), bars):
        A._within(got, r[name], bar, name)

    dnormed = (dqkv.view(n, -1).float().cpu() @ pw).cuda()
    dx, dw, db = V.layer_norm_backward(dnormed, emb, mean, rstd, weight)
    r = tower.layer_norm(_wide(emb), _wide(weight), _wide(bias), N.NORM_EPS, _wide(dnormed))
    _, _, _, dx_bar, dw_bar, db_bar = N._bars(_wide(emb), _wide(dnormed), _wide(weight), _wide(bias), r)
    N._within(dx, r["dx"], dx_bar + A.EPS * np.abs(r["dx"]), "dx")
    N._within(dw, r["dweight"], dw_bar + A.EPS * np.abs(r["dweight"]), "dweight")
    N._within(db, r["dbias"], db_bar + A.EPS * np.abs(r["dbias"]), "dbias")


def _fill(shape, seed):
    """bf16 noise of a large shape, made a slab at a time."""
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for part in t.split(1 << 17):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return t


def test_attention_past_32_bits(V):
    _say("attention of 1.1 million rows")
    length, chunks, hq, hk, d = 3520, 312, 32, 8, 64
    n = length * chunks
    assert n * hq * d > 1 << 31
    q, k, v, do = _fill((n, hq, d), 1), _fill((n, hk, d), 2), _fill((n, hk, d), 3), _fill((n, hq, d), 4)
    cu = torch.arange(chunks + 1, dtype=torch.int32, device="cuda") * length
    out, lse = V.chunk_attention(q, k, v, cu, window=64, return_lse=True)
    dq, dk, dv, _ = V.chunk_attention_backward(do, q, k, v, out, lse, cu, window=64)
    one = torch.tensor([0, length], dtype=torch.int32, device="cuda")
    for c in (0, chunks // 2, chunks - 1):
        at = slice(c * length, (c + 1) * length)
        o, l = V.chunk_attention(q[at], k[at], v[at], one, window=64, return_lse=True)
        assert torch.equal(o, out[at]) and torch.equal(l, lse[:, at])
        g = V.chunk_attention_backward(do[at], q[at], k[at], v[at], o, l, one, window=64)
        assert torch.equal(g[0], dq[at])
        # alone, a chunk's dk and dv are summed in slices: another order of the same float32 sums
        for a, b in ((g[1], dk[at]), (g[2], dv[at])):
            assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()


def test_key_gradients_past_32_bits(V):
    """dk and dv of chunks of a call of 1.1 million rows, bit for bit those of a
    call of three chunks: enough of them that neither call's sums are sliced."""
    _say("key gradients of 1.1 million rows")
    length, chunks, hq, hk, d = 3520, 312, 32, 8, 64
    n = length * chunks
    q, k, v, do = _fill((n, hq, d), 11), _fill((n, hk, d), 12), _fill((n, hk, d), 13), _fill((n, hq, d), 14)
    sink = torch.randn(hq, generator=torch.Generator().manual_seed(15)).cuda()
    cu = torch.arange(chunks + 1, dtype=torch.int32, device="cuda") * length
    out, lse = V.chunk_attention(q, k, v, cu, window=64, sink=sink, return_lse=True)
    _, dk, dv, _ = V.chunk_attention_backward(do, q, k, v, out, lse, cu, window=64, sink=sink)
    for c in (0, chunks // 2, chunks - 3):
        at = slice(c * length, (c + 3) * length)
        o, l = V.chunk_attention(q[at], k[at], v[at], cu[:4], window=64, sink=sink, return_lse=True)
        g = V.chunk_attention_backward(do[at], q[at], k[at], v[at], o, l, cu[:4], window=64, sink=sink)
        assert torch.equal(g[1], dk[at]) and torch.equal(g[2], dv[at])


def test_norm_and_product_past_32_bits(V):
    _say("norm and product of 1.7 million rows")
    n, width, e = 1_700_003, 1280, 1280
    x, do = _fill((n, width), 5), _fill((n, width), 6)
    w = torch.rand(width, generator=torch.Generator().manual_seed(7)).cuda()
    wq, ws = V.quantize_rows(torch.randn((e, width), generator=torch.Generator().manual_seed(8)).cuda())
    out, mean, rstd = V.layer_norm(x, w, w, return_stats=True)
    dx, dw, db = V.layer_norm_backward(do, x, mean, rstd, w)
    xq, xs = V.quantize_rows(x)
    y = V.quantized_linear(xq, xs, wq, ws)
    for at in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        o, m, r = V.layer_norm(x[at], w, w, return_stats=True)
        assert torch.equal(o, out[at]) and torch.equal(m, mean[at]) and torch.equal(r, rstd[at])
        assert torch.equal(V.layer_norm_backward(do[at], x[at], m, r, w)[0], dx[at])
        q, s = V.quantize_rows(x[at])
        assert torch.equal(q, xq[at]) and torch.equal(s, xs[at])
        # the kernel for few rows scales the exact sum in another order: one rounding of bf16 apart at most
        a, b = V.quantized_linear(q, s, wq, ws).float(), y[at].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs()).all()
    # dbias against sums in float64; n e sum |dout| bounds any order
    want = torch.zeros(width, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for part in do.split(1 << 17):
        want += part.double().sum(0)
        mag += part.double().abs().sum(0)
    assert ((db.double() - want).abs() <= n * 2.0 ** -24 * mag).all() and torch.isfinite(dw).all()


def test_norm_sums_and_product_rows_past_32_bits(V):
    """The weight's and bias's sums over 1.7 million rows against sums in
    float64, with a bar for the additions that there are, and the product's rows
    bit for bit the same from every kernel: blocks of 32 x 32, tiles of 128 and
    of 256."""
    _say("norm's sums and the product's rows, 1.7 million rows")
    n, width, e = 1_700_003, 1280, 1280
    x, do = _fill((n, width), 5), _fill((n, width), 6)
    w = torch.rand(width, generator=torch.Generator().manual_seed(7)).cuda()
    _, mean, rstd = V.layer_norm(x, w, w, return_stats=True)
    _, dw, db = V.layer_norm_backward(do, x, mean, rstd, w)
    _, depth = N._sums_depth(V, n, width)
    zero = lambda: torch.zeros(width, dtype=torch.float64, device="cuda")
    want_w, want_b, mag_w, mag_b, hat_bar = zero(), zero(), zero(), zero(), zero()
    rel = (width / 64 + 28 + 4 + 2) * A.EPS  # of rstd and of the distance; N._bars
    for i in range(0, n, 1 << 16):
        xx, g = x[i:i + (1 << 16)].double(), do[i:i + (1 << 16)].double()
        var, mu = torch.var_mean(xx, dim=1, unbiased=False, keepdim=True)
        hat = (xx - mu) / torch.sqrt(var + 1e-6)
        want_w += (g * hat).sum(0)
        want_b += g.sum(0)
        mag_w += (g * hat).abs().sum(0)
        mag_b += g.abs().sum(0)
        # the mean's own error, D e mean|x| with mean|x| below the spread
        hat_bar += (g.abs() * (rel * hat.abs() + (width / 64 + 20) * A.EPS)).sum(0)
    for got, want, bar in ((dw, want_w, hat_bar + depth * A.EPS * mag_w), (db, want_b, depth * A.EPS * mag_b)):
        bar = bar + A.EPS * want.abs()
        assert bar.max() < want.abs().median()  # zeros would not pass
        assert ((got.double() - want).abs() <= 1.01 * bar).all()
    del do
    wq, ws = V.quantize_rows(torch.randn((e, width), generator=torch.Generator().manual_seed(8)).cuda())
    xq, xs = V.quantize_rows(x)
    y = V.quantized_linear(xq, xs, wq, ws)
    for at in (slice(0, 300), slice(n // 2, n // 2 + 32), slice(n // 2, n // 2 + 5000), slice(n - 17, n), slice(n - 300, n)):
        assert torch.equal(V.quantized_linear(xq[at], xs[at], wq, ws), y[at])


def test_more_rows_than_a_launch_dimension_holds(V):
    """17 million rows of a width that a workgroup takes: 2^32 threads and more."""
    _say("17 million rows")
    n, width = 17_000_001, 1544
    x = torch.empty((n, width), dtype=torch.bfloat16, device="cuda")
    base = torch.randn((4096, width), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    for part in x.split(4096):
        part.copy_(base[:part.shape[0]])
    out = V.layer_norm(x, out=x)
    want = V.layer_norm(base)
    for first in (0, 4096 * 2000, 4096 * 4100, (n - 1) // 4096 * 4096):
        part = out[first:first + 4096]
        assert torch.equal(part, want[:part.shape[0]])
    del x, out
    torch.cuda.empty_cache()
