"""Plain NumPy fp64 definitions of the residual block in front of the head (matrix product with
an epilogue, dropout from a counter-based generator) and of the log-probs read off a matrix of
logits, with their gradients.

Test infrastructure only; nothing here shares code with the HIP path.
"""
import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


# ---------------------------------------------------------------- matrix product
def logistic(z):
    """1 / (1 + e^-z) to its own digits at both ends (1 + tanh(z / 2) loses those of the lower)."""
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act(z, name):
    z = np.asarray(z, np.float64)
    if name is None:
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return z * 0.5 * _erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        return z * logistic(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    assert name == "silu"
    return z * logistic(z)


def act_slope(z, name):
    z = np.asarray(z, np.float64)
    if name is None:
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        u2 = 2 * c * (z + 0.044715 * z ** 3)
        return logistic(u2) + z * logistic(u2) * logistic(-u2) * 2 * c * (1 + 3 * 0.044715 * z * z)
    assert name == "silu"
    return logistic(z) + z * logistic(z) * logistic(-z)


def linear(X, W, bias, name, residual):
    """(out, pre)"""
    pre = np.asarray(X, np.float64) @ np.asarray(W, np.float64).T
    if bias is not None:
        pre = pre + np.asarray(bias, np.float64)
    out = act(pre, name)
    return (out if residual is None else out + np.asarray(residual, np.float64)), pre


def linear_grad(dy, X, W, pre, name):
    """(dX, dW, dbias, dpre)"""
    d = np.asarray(dy, np.float64)
    if name is not None:
        d = d * act_slope(pre, name)
    return d @ np.asarray(W, np.float64), d.T @ np.asarray(X, np.float64), d.sum(axis=0), d


# ---------------------------------------------------------------- dropout
def philox(counter, key, rounds=10):
    """Philox4x32 (Salmon, Moraes, Dror, Shaw, SC11) on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_bits(M, H, seed, offset):
    out = np.empty((M, H), np.int64)
    lo = 0xFFFFFFFF
    for m in range(M):
        for b in range(-(-H // 8)):
            words = philox((b, m, offset & lo, offset >> 32), (seed & lo, seed >> 32))
            halves = [h for w in words for h in (w & 0xFFFF, w >> 16)]
            out[m, 8 * b:8 * b + 8] = halves[:H - 8 * b]
    return out


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, np.float64)
    t = int(round(65536 * p))
    keep = dropout_bits(*x.shape, seed, offset) >= t
    y = np.zeros_like(x)
    y[keep] = x[keep] / (1 - t / 65536)
    return y if residual is None else y + np.asarray(residual, np.float64)


# ---------------------------------------------------------------- log-probs from logits
def _rows(x, scale):
    """log p of every logit (NaN rows for a NaN or +inf, -inf throughout for a masked row), the
    shifted logits scale (x - max), and the log of their sum."""
    x = np.asarray(x, np.float64)
    bad = np.isnan(x).any(axis=1) | (x == np.inf).any(axis=1)
    none = (x == -np.inf).all(axis=1)
    odd = (bad | none)[:, None]
    top = np.where(odd[:, 0], 0.0, np.max(np.where(np.isnan(x), -np.inf, x), axis=1))
    with np.errstate(invalid="ignore"):
        d = scale * (np.where(odd, 0.0, x) - top[:, None])
    logs = np.log(np.exp(d).sum(axis=1))
    logp = d - logs[:, None]
    logp[none], logp[bad] = -np.inf, np.nan
    return logp, d, logs, top, bad, none


def valid_tokens(tokens, V, ignore_index):
    return (tokens != ignore_index) & (tokens >= 0) & (tokens < V)


def token_logprobs(x, tokens, ignore_index=-100, scale=1.0, n_top=0):
    """logprob, lse, entropy, top_ids, top_logprob, stats of fp64 logits; tokens [M, n]."""
    x = np.asarray(x, np.float64)
    M, V = x.shape
    logp, d, logs, top, bad, none = _rows(x, scale)
    ok = valid_tokens(tokens, V, ignore_index)
    lp = np.where(ok, np.take_along_axis(logp, np.where(ok, tokens, 0), 1), 0.0)
    lse = np.where(bad, np.nan, np.where(none, -np.inf, scale * top + logs))
    p = np.exp(np.where(np.isfinite(logp), logp, -np.inf))
    ent = -(p * np.where(p > 0, logp, 0.0)).sum(axis=1)
    ent = np.where(bad, np.nan, np.where(none, 0.0, ent))
    rank = np.where(np.isnan(x), -np.inf, x) + 0.0
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :n_top]
    with np.errstate(invalid="ignore"):
        stats = np.stack([np.where(bad, np.nan, np.where(none, -np.inf, top)), np.where(bad, np.nan, np.where(none, 0.0, logs))], 1)
    return dict(logprob=lp, lse=lse, entropy=ent, top_ids=ids, top_logprob=np.take_along_axis(logp, ids, 1), stats=stats)


def token_logprobs_grad(x, tokens, g, ignore_index=-100, scale=1.0, top_ids=None, g_top=None, g_ent=None, g_lse=None):
    x = np.asarray(x, np.float64)
    M, V = x.shape
    logp, d, logs, top, bad, none = _rows(x, scale)
    p = np.exp(logp)
    safe = np.where(p > 0, logp, 0.0)
    dx = np.zeros((M, V))
    asked = np.zeros(M, bool)
    pairs = [(tokens, g, valid_tokens(tokens, V, ignore_index))] if g is not None else []
    if g_top is not None:
        pairs.append((top_ids, g_top, np.ones(top_ids.shape, bool)))
    for t, gg, ok in pairs:
        for m in range(M):
            for j in range(t.shape[1]):
                if ok[m, j]:
                    asked[m] = True
                    dx[m] -= gg[m, j] * p[m]
                    dx[m, t[m, j]] += gg[m, j]
    if g_ent is not None:
        H = -(p * safe).sum(axis=1)
        dx -= np.asarray(g_ent)[:, None] * p * (safe + H[:, None])
        asked |= np.asarray(g_ent) != 0
    if g_lse is not None:
        dx += np.asarray(g_lse)[:, None] * p
        asked |= np.asarray(g_lse) != 0
    dx[none | ~asked] = 0.0
    return scale * dx
