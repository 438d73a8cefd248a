"""GPU parity of the rotation of query and key heads against the float64 form.
Bar: two products and a sum, each rounded to float32 (e = 2^-24), and one
rounding to bf16: 2 e (|x c| + |y s|) + 2^-8 |out|."""
import numpy as np
import pytest

import workloads as W
from oracle import tower

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS, U = 2.0 ** -24, 2.0 ** -8


def _say(*a):
    print("[gpu-rotate]", *a, flush=True)


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import vision_image_preprocessing_amd as V
    V.load()
    return V


def _wide(t):
    return t.double().cpu().numpy()


def _tables(rows, half, seed):
    angle = torch.rand((rows, half), generator=torch.Generator().manual_seed(seed)) * 300
    return angle.cos().cuda(), angle.sin().cuda()


def _noise(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _holds(got, x, cos, sin, inverse):
    want, mag = tower.rotate_heads(_wide(x), _wide(cos), _wide(sin), inverse)
    err = np.abs(_wide(got) - want)
    assert (err <= 1.01 * (2 * EPS * mag + U * np.abs(want)) + 1e-30).all(), float(err.max())


@pytest.mark.parametrize("head_dim", [8, 16, 24, 32, 64, 72, 80, 96, 128, 136, 512])
@pytest.mark.parametrize("inverse", [False, True])
def test_head_dims(V, head_dim, inverse):
    for rows, heads in ((1, 1), (3, 5), (33, 12), (7, 40)):
        _say("head_dim", head_dim, (rows, heads), inverse)
        x = _noise((rows, heads, head_dim), rows + heads)
        cos, sin = _tables(rows, head_dim // 2, rows)
        _holds(V.rotate_heads(x, cos, sin, inverse=inverse), x, cos, sin, inverse)


def test_slices_in_place_and_back(V):
    """Query and key heads as one slice of a projection's output, in place: the
    values behind them stay as they were; the inverse undoes it to two
    roundings."""
    _say("slices")
    rows, hq, hk, d = 1001, 32, 8, 64
    qkv = _noise((rows, hq + 2 * hk, d), 1)
    cos, sin = _tables(rows, d // 2, 2)
    part = qkv[:, :hq + hk]
    want = V.rotate_heads(part, cos, sin)
    assert want.is_contiguous()
    _holds(want, part, cos, sin, False)
    work = qkv.clone()
    got = V.rotate_heads(work[:, :hq + hk], cos, sin, out=work[:, :hq + hk])
    assert got.data_ptr() == work.data_ptr() and torch.equal(got, want) and torch.equal(work[:, hq + hk:], qkv[:, hq + hk:])
    back = V.rotate_heads(want, cos, sin, inverse=True)
    _holds(back, want, cos, sin, True)
    # each way rounds once: the pair's length bounds both
    length = torch.hypot(part[..., :32].double(), part[..., 32:].double()).repeat(1, 1, 2)
    assert ((back.double() - part.double()).abs() <= 2.1 * U * 2 ** 0.5 * length).all()
    # heads apart from each other, rows within a head: [heads][rows][d] in memory
    turned = part.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(V.rotate_heads(turned, cos, sin), want)
    held = torch.empty((hq + hk, rows, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(V.rotate_heads(part, cos, sin, out=held), want)


@pytest.mark.parametrize("column", [False, True])
def test_by_the_plans_tables(V, column):
    """vit_tables' cos and sin, in both orders; rows of grid position (0, 0) are not turned."""
    _say("tables", column)
    plan = V.plan_media(W.media_batch([(1, 200, 300, 3), (4, 64, 96, 3)], seed=81).items)
    t = V.vit_tables(plan, column=column)
    x = _noise((plan.total_rows, 12, 64), 3)
    got = V.rotate_heads(x, t["rope_cos"], t["rope_sin"])
    _holds(got, x, t["rope_cos"], t["rope_sin"], False)
    first = (t["rotary_pos"] == 0).all(1)
    assert first.any() and torch.equal(got[first], x[first])


def test_gradient_against_differences(V):
    """A rotation is linear: the loss's change along a direction is the inverse
    rotation's inner product with it, to the three roundings."""
    _say("differences")
    x, way, dout = _noise((50, 6, 64), 5), _noise((50, 6, 64), 6), _noise((50, 6, 64), 7)
    cos, sin = _tables(50, 32, 8)
    dx = V.rotate_heads(dout, cos, sin, inverse=True)
    moved = (x.double() + way.double()).to(torch.bfloat16)
    real = moved.double() - x.double()  # what was in fact added
    change = ((V.rotate_heads(moved, cos, sin).double() - V.rotate_heads(x, cos, sin).double()) * dout.double()).sum()
    slope = (dx.double() * real).sum()
    mag = ((moved.double().abs() + x.double().abs()).sum() + real.abs().sum()) * dout.abs().double().max() * 2 ** 0.5
    assert (change - slope).abs() <= U * mag


def test_past_32_bits(V):
    _say("past 2^31 values")
    rows, heads, d = 900_001, 40, 64
    x = torch.empty((rows, heads, d), dtype=torch.bfloat16, device="cuda")
    for i, part in enumerate(x.split(1 << 16)):
        part.copy_(_noise((257, heads, d), i).repeat(256, 1, 1)[:part.shape[0]])
    angle = torch.rand((rows, d // 2), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 100
    cos, sin = angle.cos(), angle.sin()
    out = V.rotate_heads(x, cos, sin)
    for at in (slice(0, 99), slice(rows // 2, rows // 2 + 99), slice(rows - 99, rows)):
        assert torch.equal(V.rotate_heads(x[at], cos[at], sin[at]), out[at])
        _holds(out[at], x[at], cos[at], sin[at], False)


def test_streams_graphs_and_empty(V):
    _say("streams, graphs, empty")
    x = _noise((300, 40, 64), 9)
    cos, sin = _tables(300, 32, 10)
    want = V.rotate_heads(x, cos, sin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = V.rotate_heads(x, cos, sin, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = V.rotate_heads(x, cos, sin)
    for seed in (11, 12, 13):
        x.copy_(_noise((300, 40, 64), seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, V.rotate_heads(x, cos, sin))
    none = V.rotate_heads(x[:0], cos[:0], sin[:0])
    assert none.shape == (0, 40, 64)


def test_refusals(V):
    _say("refusals")
    x = _noise((4, 3, 64), 1)
    cos, sin = _tables(4, 32, 1)
    flat = torch.zeros(4 * 3 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: V.rotate_heads(x.float(), cos, sin), lambda: V.rotate_heads(x[0], cos, sin), lambda: V.rotate_heads(x, cos[:2], sin),
                lambda: V.rotate_heads(x, cos, sin[:, :16]), lambda: V.rotate_heads(x, cos.double(), sin), lambda: V.rotate_heads(x, cos.cpu(), sin),
                lambda: V.rotate_heads(x[:, :, :60], cos, sin), lambda: V.rotate_heads(x.transpose(1, 2), cos, sin),
                lambda: V.rotate_heads(flat[1:769].view(4, 3, 64), cos, sin), lambda: V.rotate_heads(x, cos, sin, out=x[:2]),
                lambda: V.rotate_heads(x, cos, sin, out=x[:, :1].expand(4, 3, 64)),
                lambda: V.rotate_heads(x, cos, sin, out=torch.as_strided(x, (4, 3, 64), (64, 256, 1)))):
        with pytest.raises(V.MimoError):
            bad()


def test_into_other_heads_of_the_same_array(V):
    """Heads next to each other in the rows of one array are no overlap; heads
    that are, in part, those that are read are refused, and nothing is written."""
    _say("one array")
    rows, d = 500, 64
    qkv = _noise((rows, 24, d), 14)
    cos, sin = _tables(rows, d // 2, 15)
    want = V.rotate_heads(qkv[:, :8], cos, sin)
    kept = qkv.clone()
    with pytest.raises(V.MimoError, match="overlap"):
        V.rotate_heads(qkv[:, :16], cos, sin, out=qkv[:, 8:])
    with pytest.raises(V.MimoError, match="overlap"):
        V.rotate_heads(qkv[:-1], cos[:-1], sin[:-1], out=qkv[1:])
    assert torch.equal(qkv, kept)
    V.rotate_heads(qkv[:, :8], cos, sin, out=qkv[:, 16:])
    assert torch.equal(qkv[:, 16:], want) and torch.equal(qkv[:, :16], kept[:, :16])
    # every second head to the one behind it
    qkv[:, 0:16:2] = kept[:, :8]
    V.rotate_heads(qkv[:, 0:16:2], cos, sin, out=qkv[:, 1:16:2])
    assert torch.equal(qkv[:, 1:16:2], want) and torch.equal(qkv[:, 0:16:2], kept[:, :8])
    # the first rows of an array to its last ones
    V.rotate_heads(kept[:100], cos[:100], sin[:100], out=kept[400:])
    assert torch.equal(kept[400:, :8], want[:100])
