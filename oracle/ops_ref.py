"""Plain NumPy fp64 definitions of the operators around the head: layer norm and its
gradient, microscaled formats, logits and log-probs of a head with 4-bit weights.

Test infrastructure only; nothing here shares code with the HIP path.
"""
import numpy as np

BLOCK = 32


# ---------------------------------------------------------------- layer norm
def layer_norm(x, weight, bias, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    b = 0.0 if bias is None else np.asarray(bias, np.float64)
    return w * xh + b, mean, rstd


def layer_norm_grad(dy, x, mean, rstd, weight):
    """dx, dweight, dbias for given statistics (one Jacobian product a row)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64), np.asarray(rstd, np.float64)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = np.empty_like(g)
    for m in range(g.shape[0]):
        dx[m] = rstd[m] * (g[m] - g[m].mean() - xh[m] * np.mean(g[m] * xh[m]))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# ---------------------------------------------------------------- microscaled formats
def grid(fmt):
    """The non-negative values of an element format by code, ascending."""
    if fmt == "mxfp4":
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    if fmt == "mxint8":
        return np.arange(128) / 64.0
    assert fmt == "mxfp8"
    sub = [k * 2.0 ** -9 for k in range(8)]
    return np.array(sub + [(1 + k / 8) * 2.0 ** e for e in range(-6, 9) for k in range(8)][:-1])


def quantize(x, fmt):
    """(codes [rows, blocks, 32] as integers with the sign bit of the format, exponents).

    Exponent NAN_EXP marks a block that holds an infinity or a NaN (codes 0)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = np.zeros((rows, blocks * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, BLOCK)
    g = grid(fmt)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.abs(v).max(axis=2)
    exps = np.full((rows, blocks), -127)
    for e in range(-127, 127):   # the smallest exponent at which nothing exceeds the largest value
        exps = np.where((exps == e) & (top > g[-1] * 2.0 ** e), e + 1, exps)
    a = np.minimum(np.abs(v) * 2.0 ** (-exps[:, :, None].astype(np.float64)), g[-1])
    hi = np.minimum(np.searchsorted(g, a), len(g) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = g[hi] - a, a - g[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    neg = (v < 0) & (pick > 0)
    codes = np.where(neg, -pick, pick) if fmt == "mxint8" else pick + neg * len_sign(fmt)
    return codes, np.where(bad, 128, exps)


def len_sign(fmt):
    return {"mxfp4": 8, "mxfp8": 128}[fmt]


def values(codes, exps, fmt, cols):
    """The values codes and exponents stand for, [rows, cols]."""
    g = grid(fmt)
    if fmt == "mxint8":
        v = codes / 64.0
    else:
        s = len_sign(fmt)
        v = np.where(codes >= s, -1.0, 1.0) * g[codes % s]
    scale = np.where(exps == 128, np.nan, 2.0 ** np.minimum(exps, 127).astype(np.float64))
    v = v * scale[:, :, None]
    return v.reshape(v.shape[0], -1)[:, :cols]


def rounded(x, fmt):
    """The values of a matrix's microscaled copy."""
    codes, exps = quantize(x, fmt)
    return values(codes, exps, fmt, np.shape(x)[1])


# ---------------------------------------------------------------- the head in 4 bits
def fp4_logits(X, Wv, scale=1.0):
    """scale * Q(X) Wv^T with Wv the values of the quantised weights."""
    return float(np.float32(scale)) * (rounded(X, "mxfp4") @ np.asarray(Wv, np.float64).T)


def fp4_forward(X, Wv, targets, ignore_index=-100, scale=1.0):
    z = fp4_logits(X, Wv, scale)
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(axis=1)
    lse = top[:, 0] + np.log(s)
    t = np.asarray(targets)
    valid = (t != ignore_index) & (t >= 0) & (t < z.shape[1])
    zt = z[np.arange(len(t)), np.where(valid, t, 0)]
    ent = np.log(s) - (e * (z - top)).sum(axis=1) / s
    return dict(logprob=np.where(valid, zt - lse, 0.0), lse=lse,
                entropy=np.where(valid, ent, 0.0), z=z)
