"""GPU parity of rows quantised to 8 bits and of their matrix product.

quantize_rows is defined by float32 operations, each rounded correctly, so its
outputs are compared bit for bit.  The product's sum is exact; the result is
(float32(sum) * s) * t + bias: at most three roundings of e = 2^-24 of the
product, one of the sum with the bias, and the output's (u = 2^-8 for bf16, e
for float32): bar = 3.01 e |sum s t| + e (|out| + |sum s t|) + u |out|.
"""
import numpy as np
import pytest

from oracle import tower

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": EPS, "bf16": 2.0 ** -8}


def _say(*a):
    print("[gpu-quantized]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _check_quantized(V, x):
    q, s = V.quantize_rows(x.cuda())
    torch.cuda.synchronize()
    want_q, want_s = tower.quantize_rows(x.float().numpy())
    rows, width = x.shape
    assert q.shape == (rows, (width + 127) // 128 * 128)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    q = q.cpu().numpy().astype(np.int64)
    assert np.array_equal(q[:, :width], want_q) and (q[:, width:] == 0).all()


@pytest.mark.parametrize("width", [1, 2, 8, 63, 127, 128, 129, 256, 260, 512, 520, 768, 1280, 1283, 1536, 1544, 2048, 2050,
                                   5120, 6144, 6152, 9001])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_widths(V, width, kind):
    _say("quantize", width, kind)
    g = torch.Generator().manual_seed(width)
    _check_quantized(V, (torch.randn((9, width), generator=g) * 3).to(KIND[kind]))


def test_quantize_borders(V):
    """Values next to and on the border between two integers, for many scales;
    small, large, subnormal and mixed magnitudes."""
    _say("borders")
    rng = np.random.default_rng(4)
    rows = []
    for i in range(400):
        top = np.float32(rng.uniform(0.5, 2.0) * 2.0 ** rng.integers(-120, 120))
        scale = np.float32(top / np.float32(127))
        half = ((rng.integers(-126, 126, 127) + 0.5) * np.float64(scale)).astype(np.float32)
        step = rng.integers(-2, 3, 127)
        for _ in range(2):
            half = np.where(step > 0, np.nextafter(half, np.float32(np.inf)), np.where(step < 0, np.nextafter(half, np.float32(-np.inf)), half))
            step = step - np.sign(step)
        rows.append(np.concatenate([[top], half]).astype(np.float32))
    rows.append(np.float32(2.0 ** -149) * np.arange(128).astype(np.float32))
    rows.append(np.float32(2.0 ** -140) * np.arange(128).astype(np.float32))
    rows.append(np.full(128, np.float32(2.0 ** -149)))
    rows.append(np.full(128, np.finfo(np.float32).max))
    rows.append(np.zeros(128, np.float32))
    rows.append(np.where(np.arange(128) == 5, np.nan, 1.0).astype(np.float32))
    rows.append(np.where(np.arange(128) == 100, -np.inf, 1.0).astype(np.float32))
    _check_quantized(V, torch.from_numpy(np.stack(rows)))


def test_quantize_unaligned(V):
    _say("unaligned")
    x = torch.randn(5, 1280)
    s = torch.zeros(5 * 1280 + 1, device="cuda")[1:].view(5, 1280)
    s.copy_(x)
    a, b = V.quantize_rows(s), V.quantize_rows(x.cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _check_linear(V, m, n, k, out_kind, bias, seed):
    _say("linear", (m, n, k), out_kind, "bias" if bias else "")
    g = torch.Generator().manual_seed(seed)
    xq = torch.randint(-127, 128, (m, k), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(m, generator=g) * 0.02, torch.rand(n, generator=g) * 0.002
    b = torch.randn(n, generator=g) if bias else None
    out = torch.full((m + 1, n), 7.0, dtype=KIND[out_kind], device="cuda")
    V.quantized_linear(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), None if b is None else b.cuda(), out=out[:m])
    torch.cuda.synchronize()
    assert (out[m] == 7).all()
    ref, mag = tower.quantized_linear(xq.numpy(), xs.numpy(), wq.numpy(), ws.numpy(), None if b is None else b.numpy())
    bar = 3.01 * EPS * mag + EPS * (np.abs(ref) + mag) + ROUND[out_kind] * np.abs(ref)
    err = np.abs(out[:m].double().cpu().numpy() - ref)
    assert (err <= 1.01 * bar + 1e-30).all(), float((err / (bar + 1e-30)).max())


@pytest.mark.parametrize("m", [1, 2, 5, 31, 33, 64, 130])
@pytest.mark.parametrize("n", [1, 3, 32, 36, 130, 1280])
@pytest.mark.parametrize("k", [128, 384])
def test_few(V, m, n, k):
    _check_linear(V, m, n, k, "bf16" if (m + n) % 2 else "f32", n != 36, seed=m * n + k)


@pytest.mark.parametrize("m,n,k", [(2048, 1280, 1536), (2049, 1283, 256), (4100, 514, 1280), (1500, 3001, 128),
                                   (333, 8200, 640), (70000, 130, 256), (20000, 7, 128), (8200, 8200, 256),
                                   (262144, 200, 128), (32, 20000, 640), (600, 1000, 896), (1000, 300, 1408)])
@pytest.mark.parametrize("out_kind", ["f32", "bf16"])
def test_many(V, m, n, k, out_kind):
    _check_linear(V, m, n, k, out_kind, out_kind == "bf16", seed=m)


def test_longest_sums(V):
    """The widest rows of the largest magnitudes: no sum wraps."""
    _say("longest sums")
    k = 130944
    x = torch.full((2, k), 127, dtype=torch.int8)
    x[1] = -128
    w = torch.stack([torch.full((k,), 127, dtype=torch.int8), torch.full((k,), -128, dtype=torch.int8)])
    one = torch.ones(2, device="cuda")
    out = V.quantized_linear(x.cuda(), one, w.cuda(), one, out_dtype="f32").cpu().double()
    want = torch.tensor([[127 * 127, -127 * 128], [-127 * 128, 128 * 128]], dtype=torch.float64) * k
    assert (out == want.float().double()).all()


@pytest.mark.parametrize("out_kind", ["f32", "bf16"])
def test_a_row_does_not_depend_on_the_others(V, out_kind):
    """The same rows in calls of 1, 40, 300, 3000 and 70000 rows: the same bits."""
    _say("rows alone and together", out_kind)
    g = torch.Generator().manual_seed(7)
    xq = torch.randint(-127, 128, (70000, 256), generator=g, dtype=torch.int8).cuda()
    wq = torch.randint(-127, 128, (1283, 256), generator=g, dtype=torch.int8).cuda()
    xs, ws, b = torch.rand(70000, generator=g).cuda(), torch.rand(1283, generator=g).cuda(), torch.randn(1283, generator=g).cuda()
    whole = V.quantized_linear(xq, xs, wq, ws, b, out_dtype=out_kind)
    for m in (1, 40, 300, 3000):
        assert torch.equal(V.quantized_linear(xq[:m], xs[:m], wq, ws, b, out_dtype=out_kind), whole[:m]), m


@pytest.mark.parametrize("m", [2, 2000])
def test_scales_whose_product_leaves_the_range(V, m):
    """2^-100 with 2^-40, and 2^60 with 2^80 on sums of zero: the product of the
    scales alone is subnormal or infinite, the results are not.  Powers of two
    and sums below 2^24: exact."""
    _say("extreme scales", m)
    g = torch.Generator().manual_seed(8)
    xq = torch.randint(-127, 128, (m, 128), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (300, 128), generator=g, dtype=torch.int8)
    xq[1] = 0
    xs, ws = torch.full((m,), 2.0 ** -100), torch.full((300,), 2.0 ** -40)
    xs[1] = 2.0 ** 60
    wq[5], ws[5], ws[6] = 0, 2.0 ** 80, 2.0 ** -30
    want = (xq.double() @ wq.double().T) * xs.double()[:, None] * ws.double()
    out = V.quantized_linear(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out_dtype="f32").cpu()
    assert torch.isfinite(want.float()).all() and torch.equal(out, want.float())


@pytest.mark.parametrize("m", [3, 40, 300, 2000, 70000])
@pytest.mark.parametrize("out_kind", ["f32", "bf16"])
def test_row_scales_whose_product_with_a_sum_leaves_the_range(V, m, out_kind):
    """2^100 and 2^127 with small channel scales, a subnormal one among them:
    the sum times the row's scale is infinite alone, the result is not, unless
    it has to be.  Powers of two and sums below 2^24: exact in float32."""
    _say("large row scales", m, out_kind)
    g = torch.Generator().manual_seed(9)
    xq = torch.randint(-127, 128, (m, 128), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (1030, 128), generator=g, dtype=torch.int8)
    xs, ws = torch.full((m,), 0.125), torch.full((1030,), 2.0 ** -40)
    xs[0], xs[1], xs[m - 1] = 2.0 ** 100, -2.0 ** 127, 2.0 ** 64
    wq[5], ws[5], ws[7], ws[8] = 0, 2.0 ** 100, 2.0 ** 100, float("nan")
    ws[6] = 2.0 ** -149 if out_kind == "f32" else 2.0 ** -120
    want = ((xq.double() @ wq.double().T) * xs.double()[:, None] * ws.double()).float().to(KIND[out_kind])
    out = V.quantized_linear(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out_dtype=out_kind).cpu()
    assert torch.isfinite(want[:, :5]).all() and (want[0, :3] != 0).all() and torch.isinf(want[0, 7])
    assert (want[:, 5] == 0).all() and torch.isnan(out[:, 8]).all()
    keep = torch.arange(1030) != 8
    assert torch.equal(out[:, keep], want[:, keep])


def test_rows_of_large_values(V):
    """Rows up to 1e36 with weights up to 0.06, and with a bias."""
    _say("rows of large values")
    g = torch.Generator().manual_seed(10)
    for m, n in ((4, 300), (600, 1283)):
        x = (torch.rand((m, 1283), generator=g) * 2 - 0.5) * 1e36
        w, b = torch.rand((n, 1283), generator=g) * 0.06, torch.randn(n, generator=g) * 1e36
        (xq, xs), (wq, ws) = V.quantize_rows(x.cuda()), V.quantize_rows(w.cuda())
        out = V.quantized_linear(xq, xs, wq, ws, b.cuda(), out_dtype="f32").double().cpu().numpy()
        ref, mag = tower.quantized_linear(xq.cpu().numpy(), xs.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy(), b.numpy())
        assert np.abs(ref).max() < 3e38
        bar = 3.01 * EPS * mag + EPS * (np.abs(ref) + mag) + EPS * np.abs(ref)
        assert (np.abs(out - ref) <= 1.01 * bar).all()


def test_rows_that_are_not_finite(V):
    _say("not finite")
    x = torch.randn(3, 300)
    x[1, 5] = float("nan")
    w = torch.randn(40, 300)
    wq, ws = V.quantize_rows(w.cuda())
    xq, xs = V.quantize_rows(x.cuda())
    out = V.quantized_linear(xq, xs, wq, ws)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()


def test_empty(V):
    _say("empty")
    q, s = V.quantize_rows(torch.zeros((0, 100), device="cuda"))
    assert q.shape == (0, 128) and s.shape == (0,)
    wq, ws = V.quantize_rows(torch.ones((5, 100), device="cuda"))
    assert V.quantized_linear(q, s, wq, ws).shape == (0, 5)


def test_streams_and_graphs(V):
    _say("streams and graphs")
    w = torch.randn(1280, 1283, generator=torch.Generator().manual_seed(1)).cuda()
    b = torch.randn(1280).cuda()
    wq, ws = V.quantize_rows(w)
    mk = lambda s, m: torch.randn((m, 1283), generator=torch.Generator().manual_seed(s)).cuda()

    def both(x, stream=None):
        q, s = V.quantize_rows(x, stream=stream)
        return V.quantized_linear(q, s, wq, ws, b, stream=stream)

    x = mk(2, 2000)
    want = both(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(x, side)
    side.synchronize()
    assert torch.equal(got, want)
    held = []
    for m in (3, 2000):
        st = mk(3, m)
        both(st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = both(st)
        held.append((graph, st, out))
    for turn in range(3):
        for i, (graph, st, out) in enumerate(held):
            st.copy_(mk(10 + 2 * turn + i, st.shape[0]))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, both(st))
