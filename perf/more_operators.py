"""The operators of the vision tower's block that go with its attention, as they are measured: the
root-mean-square norm with the residual's addition (to bf16 or float32, to 8-bit rows, and its
training step), the rotation of query and key heads by the rotary tables, and the gated
feed-forward block with its training step.

Each case is one pass through one operator.  With ``own`` false a pass is the operator's plain
form in elementary torch operations; with ``own`` true it is the framework's call.  Rows are those
of the framework's own workloads: an image of 300x200 gives 216, one of 1024x1024 4096, a temporal
slice of a 1280x720 clip 3520; the tower has 32 query and 8 key heads of 64 and embeddings of
1280, and the feed-forward block four times as many hidden values.
"""
import math

import torch

own = False

_TYPES = {
    "f32": torch.float32,
    "bf16": torch.bfloat16,
}

NORM_EPS = 1e-6


def _norm_case(name, op, rows, width, dtype, residual=True, affine=True):
    case = {"op": op, "rows": rows, "width": width, "dtype": dtype, "residual": residual, "affine": affine}
    return {"name": name, **case} if name else case


def _rotary_case(name, rows, heads, others, head_dim, inverse=False):
    """heads: those that are rotated; others: heads of the same rows behind them (the values), which are not."""
    case = {"op": "rotary", "rows": rows, "heads": heads, "others": others, "head_dim": head_dim, "inverse": inverse}
    return {"name": name, **case} if name else case


def _mlp_case(name, op, rows, width, hidden, bias=True):
    case = {"op": op, "rows": rows, "width": width, "hidden": hidden, "bias": bias}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one small image's rows between two halves of a block: latency
        _norm_case("norm 300x200", "norm", 216, 1280, "bf16"),
        # 32 images of 1024x1024 on the way to a projection in 8 bits
        _norm_case("norm to 8 bits 32 of 1024x1024", "norm_q8", 131072, 1280, "bf16"),
        # the same rows, one step of training
        _norm_case("norm step 32 of 1024x1024", "norm_step", 131072, 1280, "bf16"),
        # float32 embeddings of an odd width, where rows are not aligned, one step of training
        _norm_case("norm step odd f32", "norm_step", 4099, 1283, "f32"),
        # one small image's queries and keys, a slice of the projection's output: latency
        _rotary_case("rotary 300x200", 216, 40, 8, 64),
        # a clip's 32 temporal slices
        _rotary_case("rotary clip", 112640, 40, 8, 64),
        # one thumbnail's rows through the feed-forward block: latency, the weights' bytes
        _mlp_case("mlp 4 rows", "mlp", 4, 1280, 5120),
        # one 300x200 image's rows: too few for the card's tiles
        _mlp_case("mlp 300x200", "mlp", 216, 1280, 5120, bias=False),
        # 32 images of 1024x1024
        _mlp_case("mlp 32 of 1024x1024", "mlp", 131072, 1280, 5120),
        # thumbnails' rows, one step of training
        _mlp_case("mlp step thumbnails", "mlp_step", 1960, 1280, 5120, bias=False),
        # odd sizes throughout, one step of training
        _mlp_case("mlp step odd", "mlp_step", 4099, 1283, 3421),
        # eight images of 1024x1024, one step of training
        _mlp_case("mlp step 8 of 1024x1024", "mlp_step", 32768, 1280, 5120),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_step", "rotary", "rotary", "mlp", "mlp", "mlp_step", "mlp_step"])
    if op.startswith("norm"):
        width = rng.choice([1280, 1280, 1024, 5120, _log(rng, 16, 9000)])
        rows = _log(rng, 1, min(131072, 131072 * 1280 // max(width, 1280)))
        return _norm_case(None, op, rows, width, rng.choice(["bf16", "f32"]), rng.random() < 0.75, rng.random() < 0.8)
    if op == "rotary":
        heads, others = rng.choice([(40, 8), (40, 8), (12, 4), (24, 0), (rng.randint(1, 32), rng.randint(0, 8))])
        head_dim = rng.choice([64, 64, 64, 32, 72, 80, 128])
        rows = _log(rng, 1, min(112640, 112640 * 48 * 64 // max((heads + others) * head_dim, 48 * 64)))
        return _rotary_case(None, rows, heads, others, head_dim, rng.random() < 0.5)
    width = rng.choice([1280, 1280, 1024, 1152, _log(rng, 8, 2200)])
    hidden = rng.choice([5120, 4 * width, 2048, _log(rng, 8, 6000)])
    most = 131072 if op == "mlp" else 32768
    rows = _log(rng, 1, min(most, most * 1280 * 5120 // max(width * hidden, 1280 * 5120)))
    return _mlp_case(None, op, rows, width, hidden, rng.random() < 0.6)


def _randn(g, shape, dtype, scale=1.0):
    """N(0, scale^2) of a type, drawn in float32."""
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    rows = case["rows"]
    if case["op"].startswith("norm"):
        width, dtype = case["width"], _TYPES[case["dtype"]]
        state["x"] = _randn(g, (rows, width), dtype)
        if case["residual"]:
            # the residual stream has channels of their own offset and spread, a few of them strong
            spread = torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 20.0, 2.0)
            offset = _randn(g, (width,), torch.float32, 0.5)
            state["residual"] = torch.addcmul(offset, torch.randn((rows, width), generator=g, device="cuda"), spread).to(dtype)
        state["weight"] = 1 + _randn(g, (width,), torch.float32, 0.2) if case["affine"] else None
        if case["op"] == "norm_step":
            state["dout"] = _randn(g, (rows, width), dtype)
            state["dresidual"] = _randn(g, (rows, width), dtype) if case["residual"] else None
        return state
    if case["op"] == "rotary":
        heads, others, d = case["heads"], case["others"], case["head_dim"]
        # rows of a projection's output: the heads that are rotated are a slice of them
        state["qkv"] = _randn(g, (rows, heads + others, d), torch.bfloat16)
        # angles as the tables have them: a patch position on a grid times the frequencies, h half and w half
        at = torch.randint(0, 256, (rows, 2), generator=g, device="cuda").float()
        half = d // 2
        freq = 1.0 / 10000.0 ** (torch.arange(0, half, 2, device="cuda").float() / half)
        angle = (at[:, :, None] * freq).reshape(rows, -1)[:, :half].contiguous()
        state["cos"], state["sin"] = angle.cos(), angle.sin()
        return state
    width, hidden = case["width"], case["hidden"]
    state["x"] = _randn(g, (rows, width), torch.bfloat16)
    state["w_gate"] = _randn(g, (hidden, width), torch.bfloat16, width ** -0.5)
    state["w_up"] = _randn(g, (hidden, width), torch.bfloat16, width ** -0.5)
    state["w_down"] = _randn(g, (width, hidden), torch.bfloat16, hidden ** -0.5)
    for name, n in (("b_gate", hidden), ("b_up", hidden), ("b_down", width)):
        state[name] = _randn(g, (n,), torch.float32, 0.1) if case["bias"] else None
    if case["op"] == "mlp_step":
        state["dout"] = _randn(g, (rows, width), torch.bfloat16)
    return state


# ---------------------------------------------------------------- plain forms

def _stream(st):
    """The rows that are normed: the sum in the residual's type, or x alone."""
    if "residual" not in st:
        return st["x"]
    return (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)


def _plain_norm(st):
    h = _stream(st)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(-1, keepdim=True) + NORM_EPS)
    hat = hf * rstd
    res = {"out": (hat if st["weight"] is None else hat * st["weight"]).to(h.dtype)}
    if "residual" in st:
        res["residual"] = h
    if st["case"]["op"] == "norm_step":
        dy = st["dout"].float()
        gr = dy if st["weight"] is None else dy * st["weight"]
        dx = rstd * (gr - hat * (gr * hat).mean(-1, keepdim=True))
        if st["dresidual"] is not None:
            dx = dx + st["dresidual"].float()
        res["dx"] = dx.to(h.dtype)
        if st["weight"] is not None:
            res["dweight"] = (dy * hat).sum(0, dtype=torch.float64).float()
    return res


def _plain_norm_q8(st):
    h = _stream(st)
    hf = h.float()
    # in 64 bits: a value next to the middle of two integers goes by the last bit of rstd
    square = hf.double().square_().mean(-1, keepdim=True)
    y = hf * (1.0 / torch.sqrt(square + NORM_EPS)).float()
    if st["weight"] is not None:
        y = y * st["weight"]
    # divisions, which products with the constant's reciprocal are not
    scale = y.abs().amax(1) / torch.full((1,), 127.0, device=y.device)
    q = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None]).to(torch.int8)
    res = {"q": q, "scale": scale}
    if "residual" in st:
        res["residual"] = h
    return res


def _plain_rotary(st):
    case = st["case"]
    half = case["head_dim"] // 2
    x = st["qkv"][:, :case["heads"]].float()
    a, b = x[..., :half], x[..., half:]
    c, s = st["cos"][:, None], st["sin"][:, None]
    if case["inverse"]:
        s = -s
    return {"out": torch.cat((a * c - b * s, b * c + a * s), -1).to(torch.bfloat16)}


def _affine(x, w, b):
    y = torch.matmul(x, w.float().t())
    return y if b is None else y + b


def _plain_mlp(st):
    x = st["x"].float()
    gate, up = _affine(x, st["w_gate"], st["b_gate"]), _affine(x, st["w_up"], st["b_up"])
    sig = torch.sigmoid(gate)
    act = gate * sig
    hidden = act * up
    res = {"out": _affine(hidden, st["w_down"], st["b_down"]).to(torch.bfloat16)}
    if st["case"]["op"] == "mlp":
        return res
    dy = st["dout"].float()
    dh = torch.matmul(dy, st["w_down"].float())
    dgate = dh * up * (sig * (1.0 + gate * (1.0 - sig)))
    dup = dh * act
    dx = torch.matmul(dgate, st["w_gate"].float()) + torch.matmul(dup, st["w_up"].float())
    res["dx"] = dx.to(torch.bfloat16)
    for name, left, right in (("dw_gate", dgate, x), ("dw_up", dup, x), ("dw_down", dy, hidden)):
        res[name] = torch.matmul(left.t(), right).to(torch.bfloat16)
    if st["case"]["bias"]:
        for name, t in (("db_gate", dgate), ("db_up", dup), ("db_down", dy)):
            res[name] = t.sum(0, dtype=torch.float64).float()
    return res


# ---------------------------------------------------------------- one pass

def _own_norm(V, st):
    op, residual = st["case"]["op"], st.get("residual")
    if op == "norm_q8":
        got = V.rms_norm_quantized(st["x"], st["weight"], residual, eps=NORM_EPS)
        # rows of q are padded with zeros
        res = {"q": got[0][:, :st["case"]["width"]], "scale": got[1]}
        if residual is not None:
            res["residual"] = got[2]
        return res
    got = V.rms_norm(st["x"], st["weight"], residual, eps=NORM_EPS, return_rstd=op == "norm_step")
    if op == "norm":
        return {"out": got} if residual is None else {"out": got[0], "residual": got[1]}
    res = {"out": got[0]}
    normed = st["x"]
    if residual is not None:
        normed = res["residual"] = got[1]
    dx, dweight = V.rms_norm_backward(st["dout"], normed, got[-1], st["weight"], dresidual=st["dresidual"])
    res["dx"] = dx
    if dweight is not None:
        res["dweight"] = dweight
    return res


def _own_pass(st):
    import vision_image_preprocessing_amd as V
    case = st["case"]
    if case["op"].startswith("norm"):
        return _own_norm(V, st)
    if case["op"] == "rotary":
        return {"out": V.rotate_heads(st["qkv"][:, :case["heads"]], st["cos"], st["sin"], inverse=case["inverse"])}
    weights, biases = (st["w_gate"], st["w_up"], st["w_down"]), (st["b_gate"], st["b_up"], st["b_down"])
    if case["op"] == "mlp":
        return {"out": V.gated_mlp(st["x"], *weights, *biases)}
    out, gate_up, hidden = V.gated_mlp(st["x"], *weights, *biases, return_saved=True)
    grads = V.gated_mlp_backward(st["dout"], st["x"], *weights, gate_up, hidden, bias_grads=case["bias"])
    names = ("dx", "dw_gate", "dw_up", "dw_down", "db_gate", "db_up", "db_down")
    return {"out": out, **{n: t for n, t in zip(names, grads) if t is not None}}


def run(state):
    if own:
        return _own_pass(state)
    op = state["case"]["op"]
    if op == "norm_q8":
        return _plain_norm_q8(state)
    if op.startswith("norm"):
        return _plain_norm(state)
    return _plain_rotary(state) if op == "rotary" else _plain_mlp(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, rows = case["op"], case["rows"]
    if op.startswith("norm"):
        n, size = rows * case["width"], 4 if case["dtype"] == "f32" else 2
        weight = case["width"] * 4 if case["affine"] else 0
        # x (and the residual) in, out (and the residual) out
        stream = n * size * (3 if case["residual"] else 1)
        if op == "norm_q8":
            return {"bytes": stream + n + 4 * rows + weight, "flops": 8 * n}
        if op == "norm":
            return {"bytes": stream + n * size + weight, "flops": 5 * n}
        # and dout (and the residual's gradient) in, dx out; dweight out
        return {"bytes": stream + n * size * (4 if case["residual"] else 3) + 2 * weight, "flops": 16 * n}
    if op == "rotary":
        n = rows * case["heads"] * case["head_dim"]
        return {"bytes": 4 * n + rows * case["head_dim"] * 4, "flops": 3 * n}
    d, h = case["width"], case["hidden"]
    weights = 6 * d * h
    if op == "mlp":
        return {"bytes": 4 * rows * d + weights, "flops": 6 * rows * d * h}
    # x, dout and the weights in, out, dx and the weights' gradients out
    return {"bytes": 8 * rows * d + 2 * weights, "flops": 18 * rows * d * h}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_norm(case, st):
    wide = st["x"].double()
    if case["residual"]:
        # the stream is held in its type: the norm is that of the rounded sum (a float32 sum of values of that type)
        kept = torch.add(st["x"].float(), st["residual"].float()).to(st["residual"].dtype)
        wide = kept.double()
    n = case["width"]
    inv = (torch.linalg.vector_norm(wide, dim=1).square() / n + NORM_EPS).pow(-0.5)
    w = torch.ones(n, dtype=torch.float64, device="cuda") if st["weight"] is None else st["weight"].double()
    if case["op"] == "norm_q8":
        # by definition both products and both quotients are rounded to float32, and the last goes to the nearest
        # whole number, a tie to even
        y = (wide * inv.float().double()[:, None]).float()
        y = (y.double() * w).float()
        scale = (y.abs().amax(1).double() / 127.0).float()
        q = (y.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]).float().double().round()
        res = {"q": q.to(torch.int8), "scale": scale.double()}
    else:
        res = {"out": wide * inv[:, None] * w}
    if case["residual"]:
        res["residual"] = wide
    if case["op"] == "norm_step":
        dy = st["dout"].double()
        dhat = dy * w
        # d/dh of h (h.h / n + eps)^-1/2
        dx = dhat * inv[:, None] - wide * ((dhat * wide).sum(1) * inv.pow(3) / n)[:, None]
        res["dx"] = dx if st["dresidual"] is None else dx + st["dresidual"].double()
        if st["weight"] is not None:
            res["dweight"] = torch.einsum("rc,r->c", dy * wide, inv)
    return res


def _exact_rotary(case, st):
    d = case["head_dim"]
    x = st["qkv"][:, :case["heads"]].double()
    z = torch.complex(x[..., :d // 2], x[..., d // 2:])
    turn = torch.complex(st["cos"].double(), st["sin"].double())[:, None]
    z = z * (turn.conj() if case["inverse"] else turn)
    return {"out": torch.cat((z.real, z.imag), -1)}


def _exact_mlp(case, st):
    def zero(n):
        return torch.zeros(n, dtype=torch.float64, device="cuda")

    bg, bu, bd = (zero(n) if st[k] is None else st[k].double() for k, n in
                  (("b_gate", case["hidden"]), ("b_up", case["hidden"]), ("b_down", case["width"])))
    wg, wu, wd = st["w_gate"].double(), st["w_up"].double(), st["w_down"].double()
    step = case["op"] == "mlp_step"
    parts = {"out": [], "dx": []}
    sums = {k: torch.zeros_like(t) for k, t in (("dw_gate", wg), ("dw_up", wu), ("dw_down", wd), ("db_gate", bg), ("db_up", bu), ("db_down", bd))}
    for r in range(0, case["rows"], 16384):
        x = st["x"][r:r + 16384].double()
        a, b = torch.addmm(bg, x, wg.T), torch.addmm(bu, x, wu.T)
        s = 1.0 / (1.0 + torch.exp(-a))
        h = a * s * b
        parts["out"].append(torch.addmm(bd, h, wd.T))
        if not step:
            continue
        dy = st["dout"][r:r + 16384].double()
        dh = dy @ wd
        da, db = dh * b * (s + a * s * (1.0 - s)), dh * a * s
        parts["dx"].append(torch.addmm(da @ wg, db, wu))
        for k, t in (("dw_gate", da.T @ x), ("dw_up", db.T @ x), ("dw_down", dy.T @ h), ("db_gate", da.sum(0)),
                     ("db_up", db.sum(0)), ("db_down", dy.sum(0))):
            sums[k] += t
    if not step:
        return {"out": torch.cat(parts["out"])}
    return {**{k: torch.cat(v) for k, v in parts.items()}, **{k: v for k, v in sums.items() if case["bias"] or k.startswith("dw")}}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    return _exact_rotary(case, st) if case["op"] == "rotary" else _exact_mlp(case, st)
