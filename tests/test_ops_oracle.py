"""Pins of the fp64 definitions in oracle/ops_ref.py: closed forms, finite differences and
brute force."""
import numpy as np
import pytest

from oracle import ops_ref as ops


def test_layer_norm_closed_form():
    y, mean, rstd = ops.layer_norm([[1.0, 3.0]], [2.0, 1.0], [0.5, 0.0], 0.0)
    assert mean[0] == 2.0 and rstd[0] == 1.0
    assert np.allclose(y, [[-1.5, 1.0]])
    # a constant row: nothing but the bias
    y, _, rstd = ops.layer_norm([[7.0, 7.0, 7.0]], None, [1.0, 2.0, 3.0], 0.25)
    assert np.allclose(y, [[1.0, 2.0, 3.0]]) and rstd[0] == 2.0


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(11)
    x, dy = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    w, b, eps = rng.standard_normal(7), rng.standard_normal(7), 1e-3
    _, mean, rstd = ops.layer_norm(x, w, b, eps)
    dx, dw, db = ops.layer_norm_grad(dy, x, mean, rstd, w)
    f = lambda x_, w_, b_: float((ops.layer_norm(x_, w_, b_, eps)[0] * dy).sum())
    h = 1e-6

    def diff(args, k):
        out = np.empty(args[k].size)
        for i in range(args[k].size):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[k].flat[i] -= h
            hi[k].flat[i] += h
            out[i] = (f(*hi) - f(*lo)) / (2 * h)
        return out.reshape(args[k].shape)

    for got, k in ((dx, 0), (dw, 1), (db, 2)):
        assert np.allclose(got, diff((x, w, b), k), atol=1e-7)


@pytest.mark.parametrize("fmt, n", [("mxfp4", 8), ("mxfp8", 127), ("mxint8", 128)])
def test_grids(fmt, n):
    g = ops.grid(fmt)
    assert len(g) == n and np.all(np.diff(g) > 0) and g[0] == 0
    assert g[-1] == {"mxfp4": 6.0, "mxfp8": 448.0, "mxint8": 127 / 64}[fmt]


def test_fp8_grid_is_torchs_e4m3():
    import torch
    g = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(g, ops.grid("mxfp8"))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "mxint8"])
def test_quantize_by_brute_force(fmt):
    rng = np.random.default_rng(12)
    x = (rng.standard_normal((6, 70)) * 10.0 ** rng.integers(-3, 4, (6, 70))).astype(np.float32)
    x[0, :32] = 0
    q = ops.rounded(x, fmt)
    g = ops.grid(fmt)
    both = np.concatenate([-g[::-1], g])
    for r in range(6):
        for b in range(3):
            block = x[r, 32 * b:32 * b + 32].astype(np.float64)
            fits = [e for e in range(-127, 128) if np.all(np.abs(block) <= g[-1] * 2.0 ** e)]
            grid = both * 2.0 ** fits[0]
            for i, v in enumerate(block):
                best = np.abs(grid - v).min()
                assert abs(q[r, 32 * b + i] - v) == best


def test_quantize_ties_and_values():
    x = np.zeros((1, 32))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    assert ops.rounded(x, "mxfp4")[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4]
    x[0, 0] = 6.5   # the next scale
    assert ops.rounded(x, "mxfp4")[0, :3].tolist() == [6, 0, 1]
    x[0, 3] = np.inf
    assert np.isnan(ops.rounded(x, "mxfp4")).all()


def test_fp4_forward_matches_log_softmax():
    import torch
    rng = np.random.default_rng(13)
    X, W = rng.standard_normal((5, 64)), rng.standard_normal((40, 64))
    t = np.array([3, -100, 39, 40, 0])
    o = ops.fp4_forward(X, W, t, scale=0.5)
    z = 0.5 * ops.rounded(X, "mxfp4") @ W.T
    lp = torch.log_softmax(torch.from_numpy(z), 1).numpy()
    assert np.allclose(o["logprob"], [lp[0, 3], 0, lp[2, 39], 0, lp[4, 0]])
    e = -(np.exp(lp) * lp).sum(1)
    assert np.allclose(o["entropy"], e * [1, 0, 1, 0, 1])
