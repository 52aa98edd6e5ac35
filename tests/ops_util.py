"""Helpers of the tests of layer norm and microscaled formats: packing of codes, and error
bounds counted from the roundings of each path."""
import numpy as np

U32 = 2.0 ** -24   # half a step of fp32
U16 = 2.0 ** -8    # half a step of bf16


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def pack(codes, fmt):
    """Integer codes [rows, blocks, 32] as the bytes of a row."""
    rows = codes.shape[0]
    c = codes.reshape(rows, -1).astype(np.int64)
    if fmt == "mxfp4":
        return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    return (c & 255).astype(np.uint8)


def pack_scales(exps):
    rows, blocks = exps.shape
    out = np.zeros((rows, -(-blocks // 16) * 16), np.uint8)
    out[:, :blocks] = exps + 127
    return out


def norm_depth(H):
    """Additions a value passes through in a row's sum: a thread holds at most H / 64 of the
    elements, or 8 in the rows of fewer threads, then the lanes and waves."""
    return H / 64 + 40


def norm_forward_bounds(x, weight, bias, eps, y, mean, rstd, half):
    """Elementwise error bounds of (y, mean, rstd) in 32-bit arithmetic, y rounded with `half`
    relative.  x etc. are the fp64 values."""
    H = x.shape[1]
    K = norm_depth(H)
    w = 1.0 if weight is None else np.abs(weight)
    e_mean = (K + 2) * U32 * np.abs(x).mean(axis=1)
    var = 1.0 / rstd ** 2 - eps
    # the centred squares: their sum's own roundings, and the shift by the mean's error
    rel = 0.5 * ((K + 8) * U32 * np.maximum(var, 0) + e_mean ** 2) * rstd ** 2 + 4 * U32
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    e_xh = xh * (rel[:, None] + 4 * U32) + (e_mean * rstd)[:, None] * (1 + rel[:, None])
    e_y = w * e_xh + 3 * U32 * (w * xh + (0 if bias is None else np.abs(bias)))
    return (half * (np.abs(y) + e_y) + e_y, e_mean, rstd * rel)


def norm_backward_bounds(dy, x, mean, rstd, weight, dx, dw, db, half_x, half_p):
    """Elementwise bounds of (dx, dweight, dbias) for given statistics."""
    M, H = x.shape
    K = norm_depth(H)
    D = M / 256 + 100   # additions over rows: a group's rows, then the groups' partial sums
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy) * (1.0 if weight is None else np.abs(weight))
    mg = g.mean(axis=1, keepdims=True)
    mgx = (g * xh).mean(axis=1, keepdims=True)
    e = rstd[:, None] * (6 * U32 * (g + mg + xh * mgx) + (K + 4) * U32 * mg + xh * (K + 8) * U32 * mgx)
    e_w = (D + 6) * U32 * (np.abs(dy) * xh).sum(axis=0)
    e_b = (D + 4) * U32 * np.abs(dy).sum(axis=0)
    return (half_x * (np.abs(dx) + e) + e, half_p * (np.abs(dw) + e_w) + e_w,
            half_p * (np.abs(db) + e_b) + e_b)


def check_within(got, want, bound, label):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, label
    assert np.isfinite(got).all(), f"{label}: not finite"
    over = np.abs(got - want) - bound - 1e-38
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else ()
    assert not over.size or over[worst] <= 0, (
        f"{label}: at {worst} got {got[worst]!r}, expected {want[worst]!r}, "
        f"bound {np.broadcast_to(bound, got.shape)[worst]!r}")
