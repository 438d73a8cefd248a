"""Plain float64 forms of the vision tower's operators (NumPy, one chunk, head
or row at a time), written from their formulas and sharing no code with the
HIP library."""
from __future__ import annotations

import numpy as np


def _logits(q, k, window, scale, sink):
    s = scale * (q @ k.T)
    s[:, 0] += sink
    if window is not None and window >= 0:
        i = np.arange(q.shape[0])
        s[np.abs(i[:, None] - i[None, :]) > window] = -np.inf
    return s


def _softmax(s):
    """(probabilities, log of the sum); a row of -inf gives zeros and -inf."""
    top = s.max(axis=1)
    safe = np.where(np.isneginf(top), 0.0, top)
    e = np.exp(s - safe[:, None])
    total = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = safe + np.log(total)
    return e / np.where(total > 0, total, 1.0)[:, None], lse


def chunk_attention(q, k, v, cu, window=-1, scale=None, sink=None, dout=None):
    """q [rows, hq, d], k and v [rows, hk, d] (float64); cu: boundaries.

    Returns a dict: out, lse [hq, rows] (rows of no chunk: zeros), and with
    dout also dq, dk, dv, dsink, plus the sums of magnitudes that error bounds
    are made of (keys starting with "abs_")."""
    rows, hq, d = q.shape
    hk = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    r = {"out": np.zeros_like(q), "lse": np.zeros((hq, rows)), "seen": np.zeros((hq, rows)),
         "abs_s": np.zeros((hq, rows)), "abs_out": np.zeros_like(q)}
    if dout is not None:
        r.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dsink=np.zeros(hq))
    r["parts"] = []
    for a, b in zip(cu[:-1], cu[1:]):
        if b <= a:
            continue
        for h in range(hq):
            g = h // (hq // hk)
            qh, kh, vh = q[a:b, h], k[a:b, g], v[a:b, g]
            s = _logits(qh, kh, window, scale, 0.0 if sink is None else sink[h])
            p, lse = _softmax(s)
            r["out"][a:b, h] = p @ vh
            r["lse"][h, a:b] = lse
            r["seen"][h, a:b] = np.isfinite(s).sum(axis=1)
            r["abs_s"][h, a:b] = scale * (np.abs(qh) @ np.abs(kh).T).max(axis=1) + (0.0 if sink is None or np.isinf(sink[h]) else abs(sink[h]))
            r["abs_out"][a:b, h] = p @ np.abs(vh)
            if dout is None:
                continue
            do = dout[a:b, h]
            dp = do @ vh.T
            delta = (do * r["out"][a:b, h]).sum(axis=1)
            ds = p * (dp - delta[:, None])
            r["dq"][a:b, h] = scale * ds @ kh
            r["dk"][a:b, g] += scale * ds.T @ qh
            r["dv"][a:b, g] += p.T @ do
            r["dsink"][h] += ds[:, 0].sum()
            r["parts"].append((a, b, h, g, p, dp, ds))
    return r


def layer_norm(x, weight, bias, eps, dout=None):
    """x [rows, n] (float64), weight and bias [n] or None.

    Returns a dict: out, mean, rstd, hat, and with dout dx, dweight, dbias."""
    n = x.shape[1]
    mean = x.sum(axis=1) / n
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / n + eps)
    hat = d * rstd[:, None]
    w = np.ones(n) if weight is None else weight
    r = {"out": hat * w + (0.0 if bias is None else bias), "mean": mean, "rstd": rstd, "hat": hat}
    if dout is not None:
        g = dout * w
        s1, s2 = g.sum(axis=1) / n, (g * hat).sum(axis=1) / n
        r.update(dx=rstd[:, None] * (g - s1[:, None] - hat * s2[:, None]), dweight=(dout * hat).sum(axis=0),
                 dbias=dout.sum(axis=0), g=g, s1=s1, s2=s2)
    return r


def quantize_rows(x):
    """(q int64 [rows, n], scale float32 [rows]) of float32 rows, by the
    definition: both quotients are float32 divisions."""
    x = np.asarray(x, dtype=np.float32)
    top = np.abs(x).max(axis=1)
    finite = np.isfinite(x).all(axis=1)
    scale = np.where(finite, top / np.float32(127.0), np.float32(np.nan)).astype(np.float32)
    usable = finite & (scale > 0)
    q = np.zeros(x.shape, dtype=np.int64)
    q[usable] = np.clip(np.rint(x[usable] / scale[usable][:, None]), -127, 127).astype(np.int64)
    return q, scale


def quantized_linear(xq, x_scale, wq, w_scale, bias=None):
    """(out, |sum| scaled) in float64, from exact integer sums."""
    total = (np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T)
    s = np.asarray(x_scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)[None, :]
    out = total * s
    return (out if bias is None else out + np.asarray(bias, dtype=np.float64)), np.abs(total * s)
