"""Error bounds of the residual block's kernels and of the log-probs from logits, counted from
the roundings of the 32-bit paths."""
import numpy as np

from oracle import block_ref as ref
from tests.ops_util import U16, U32


def product_depth(K):
    """Roundings that a term of a dot product of K passes through: the matrix instruction adds 16 at
    a time (four or five levels, each perhaps cut rather than rounded: two half steps), then shares
    of a split K, bias and the store."""
    return 2 * (K / 16 + 5) + 40


def act_error(z, name):
    """Bound of the fp32 activation's own error at z."""
    z = np.asarray(z, np.float64)
    a = np.abs(ref.act(z, name))
    if name in (None, "relu"):
        return 0 * z
    if name == "gelu":
        # polynomial 4e-7 < 2^-21, the exponential's argument z^2 / 2 twice rounded, a few more
        q = np.abs(z) * ref.act(-np.abs(z), "gelu") / np.where(z == 0, 1, -np.abs(z))
        return np.abs(q) * (2.0 ** -20 + z * z * 2 * U32) + 4 * U32 * a
    u = np.abs(z) if name == "silu" else 1.6 * np.abs(z) * (1 + 0.045 * z * z)
    # the logistic function: relative to its value, the error of its argument and of exp and rcp
    return a * (2.0 ** -21 + 6 * U32 * np.minimum(u, 100))


def slope_error(z, name):
    """Bound of the fp32 slope's own error (slopes are at most 1.13 in magnitude)."""
    z = np.asarray(z, np.float64)
    if name in (None, "relu"):
        return 0 * z
    c = np.minimum(np.abs(z), 30)
    tail = np.exp(-np.minimum(c, 20))   # both Phi's tail and the logistic's are below it past 2
    return 2.0 ** -20 + (1 + c ** 4) * tail * 16 * U32


def linear_bounds(X, W, bias, name, residual, half):
    """Bounds of (out, pre) for fp64 arrays of the operands' values."""
    out, pre = ref.linear(X, W, bias, name, residual)
    mag = np.abs(X) @ np.abs(W).T + (0 if bias is None else np.abs(bias))
    e_pre = product_depth(X.shape[1]) * U32 * mag
    e = 1.2 * e_pre + act_error(pre, name) + 1.2 * act_error(pre + e_pre, name)
    if residual is not None:
        e = e + U32 * (np.abs(out) + np.abs(residual))
    return out, pre, half * (np.abs(out) + e) + e, U16 * (np.abs(pre) + e_pre) + e_pre


def linear_grad_bounds(dy, X, W, pre, name, rounded):
    """(want, bound) pairs of dX, dW, dbias; `rounded`: dpre goes through bf16."""
    dx, dw, db, d = ref.linear_grad(dy, X, W, pre, name)
    M, N = d.shape
    e_d = np.abs(dy) * slope_error(pre, name) + 2 * U32 * np.abs(d) if name else 0 * d
    e_r = e_d + (U16 * (np.abs(d) + e_d) if rounded else 0)
    mag = np.abs(d) + e_r
    e_x = e_r @ np.abs(W) + product_depth(N) * U32 * (mag @ np.abs(W))
    e_w = e_r.T @ np.abs(X) + product_depth(M) * U32 * (mag.T @ np.abs(X))
    # a column's sum: a wave's rows, then the groups'
    e_b = e_d.sum(axis=0) + (M / 4 + 200) * U32 * np.abs(d).sum(axis=0)
    return [(dx, U16 * (np.abs(dx) + e_x) + e_x), (dw, U16 * (np.abs(dw) + e_w) + e_w), (db, e_b)]


def sum_error(x, scale, V):
    """Bounds of log S and of U / S (the mean shift, natural units) of rows of finite or masked
    logits, absolute."""
    logp, d, logs, top, bad, none = ref._rows(x, scale)
    p = np.exp(np.where(np.isfinite(logp), logp, -np.inf))
    ad = np.where(p > 0, np.abs(d), 0.0)
    depth = V / 2048 + 60      # a thread's vectors, lanes, waves, pieces of a row
    rel = 8 * U32 + 4 * U32 * ad   # an exponential: its own error and its argument's
    e_s = (p * rel).sum(axis=1) + depth * U32
    e_u = (p * ad * (rel + 4 * U32)).sum(axis=1) + depth * U32 * (p * ad).sum(axis=1) + e_s * (p * ad).sum(axis=1)
    return e_s, e_u


def logprob_error(want, logs, e_s, x_scaled):
    """Bound of a log-prob: its shifted logit's and the log's roundings."""
    return e_s + 4 * U32 * (np.abs(x_scaled) + np.abs(logs)) + U32 * np.abs(want)
