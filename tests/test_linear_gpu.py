"""The matrix product with an epilogue and its gradient on the GPU against the fp64 definition,
with bounds counted from the roundings of each path (tests/block_util.py)."""
import numpy as np
import pytest

from oracle import block_ref as ref
from tests import block_util as bu
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def make(M, N, K, seed, bias="fp32", residual=None, spread=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return dict(X=n(M, K).bfloat16(), W=(spread * n(N, K) / K ** 0.5).bfloat16(),
                b=None if bias is None else (0.3 * n(N)).to(dt(bias)),
                r=None if residual is None else n(M, N).to(dt(residual)), dy=n(M, N))


def f64(t):
    return None if t is None else ou.np64(t)


def check_forward(s, act, out, label, keep=True):
    from log_prob_amd import flce
    want, pre64, e_out, e_pre = bu.linear_bounds(f64(s["X"]), f64(s["W"]), f64(s["b"]), act, f64(s["r"]),
                                                 ou.half_step(dt(out)))
    y = flce.linear_forward(s["X"], s["W"], s["b"], act, s["r"], dt(out), keep)
    y, pre = y if keep else (y, None)
    assert y.dtype == dt(out)
    ou.check_within(ou.np64(y), want, e_out, f"{label} out")
    if keep:
        ou.check_within(ou.np64(pre), pre64, e_pre, f"{label} pre")
    return y, pre


def check_backward(s, act, pre, dy, bias, label):
    import torch
    from log_prob_amd import flce
    got = flce.linear_backward(dy, s["X"], s["W"], pre, act, bias_dtype=bias)
    rounded = act is not None or dy.dtype == torch.float32
    pairs = bu.linear_grad_bounds(f64(dy), f64(s["X"]), f64(s["W"]), f64(pre), act, rounded)
    for name, g, (want, bound) in zip(("dX", "dW", "dbias"), got, pairs):
        if g is None:
            assert name == "dbias" and bias is None
            continue
        if name == "dbias":
            assert g.dtype == bias
            bound = ou.half_step(bias) * (np.abs(want) + bound) + bound
        else:
            assert g.dtype == torch.bfloat16
        ou.check_within(ou.np64(g), want, bound, f"{label} {name}")
    return got


# one row to many; every tile and split; odd widths; K of one step and less
SHAPES = [(1, 1, 8), (1, 17, 64), (2, 130, 72), (3, 64, 2048), (5, 100, 520), (8, 33, 4104), (9, 48, 64), (16, 4096, 512),
          (31, 257, 200), (64, 64, 64), (64, 200, 4096), (65, 128, 128), (100, 1000, 1000), (129, 300, 2056),
          (257, 1031, 136), (300, 72, 8), (513, 640, 192)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K):
    import torch
    for i, act in enumerate(ACTS):
        out = ("bf16", "fp32")[(i + M) % 2]
        s = make(M, N, K, M + N + K + i, bias=(None, "fp32", "bf16")[(i + N) % 3],
                 residual=(None, "fp32", "bf16")[(i + M + N) % 3])
        y, pre = check_forward(s, act, out, f"{M}x{N}x{K} {act}")
        dy = s["dy"].to(dt(("fp32", "bf16")[i % 2]))
        check_backward(s, act, pre, dy, (torch.float32, torch.bfloat16, None)[i % 3], f"{M}x{N}x{K} {act}")


# where one kernel hands over to the next: dot products, W streamed for 16 and 32 rows, tiles
EDGES = [(2, 4099, 1032), (3, 16, 8), (16, 17, 520), (17, 4100, 512), (20, 33, 1032), (32, 15, 4096), (32, 8200, 64),
         (33, 130, 2048), (4, 40000, 72), (30, 60001, 136), (192, 16500, 320), (260, 20000, 1600)]


@pytest.mark.parametrize("M,N,K", EDGES)
def test_edges_between_kernels(M, N, K):
    for i, (act, res) in enumerate((("gelu", "fp32"), (None, "bf16"))):
        check_forward(make(M, N, K, M + N + K + i, bias="bf16", residual=res), act, ("fp32", "bf16")[i],
                      f"{M}x{N}x{K} {act}")


# a last tile row of half the height or less, of just more, and one of a split K; tiles of 128 and 256
@pytest.mark.parametrize("M,N,K", [(1025, 4096, 72), (320, 9001, 1024), (577, 4100, 1032), (300, 4090, 4096),
                                   (513, 20001, 328), (2176, 4096, 256), (2177, 4099, 256)])
def test_last_tile_row(M, N, K):
    for i, (act, res) in enumerate((("silu", "bf16"), (None, "fp32"))):
        check_forward(make(M, N, K, 2 * M + N + K + i, bias="fp32", residual=res), act, ("bf16", "fp32")[i],
                      f"{M}x{N}x{K} {act}")


# dX of few rows and values, and just past them; N of one share, a ragged one and many
@pytest.mark.parametrize("M,N,K", [(1, 37832, 104), (1, 1, 1024), (4, 50257, 256), (3, 129, 336), (2, 3000, 512),
                                   (1, 130, 1032), (4, 4096, 264), (1, 20001, 8)])
def test_gradient_of_few_values(M, N, K):
    import torch
    for i, act in enumerate(("silu", None)):
        s = make(M, N, K, 3 * M + N + K + i, bias="fp32")
        y, pre = check_forward(s, act, "bf16", f"{M}x{N}x{K} {act}")
        for dy in (s["dy"].float(), s["dy"].bfloat16()):
            check_backward(s, act, pre, dy, torch.float32, f"{M}x{N}x{K} {act} {dy.dtype}")


@pytest.mark.parametrize("M,N,K,act", [(4096, 4096, 256, "gelu"), (3000, 5003, 320, None), (4100, 3900, 72, "silu")])
def test_large_tiles(M, N, K, act):
    import torch
    s = make(M, N, K, 7, residual="bf16")
    y, pre = check_forward(s, act, "bf16", "large")
    check_backward(s, act, pre, s["dy"].bfloat16(), torch.float32, "large")


@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_over_their_range(act):
    """From -30 to 30 and beyond, through the forward and the slope (M = 1 and a tile)."""
    import torch
    from log_prob_amd import flce
    z = torch.cat([torch.linspace(-30, 30, 1991), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 100.0, -100.0, 1e4, -1e4,
                                                                1e20])]).float().cuda()
    for M in (1, 40):
        X, W = torch.zeros(M, 8, device="cuda").bfloat16(), torch.zeros(2000, 8, device="cuda").bfloat16()
        y = flce.linear_forward(X, W, z, act, out_dtype=torch.float32)
        z64 = ou.np64(z)
        ou.check_within(ou.np64(y), np.broadcast_to(ref.act(z64, act), (M, 2000)),
                        bu.act_error(z64, act) + 1e-37, f"{act} {M}")
        pre = z.bfloat16().expand(M, 2000).contiguous()
        dy = torch.ones(M, 2000, device="cuda")
        db = flce.linear_backward(dy, X, W, pre, act, False, False, torch.float32)[2]
        p64 = ou.np64(pre[0])
        ou.check_within(ou.np64(db) / M, ref.act_slope(p64, act),
                        bu.slope_error(p64, act) + 200 * ou.U32 * np.abs(ref.act_slope(p64, act)), f"{act} slope {M}")


@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_nonfinite_values_stay_in_their_rows(M):
    import torch
    from log_prob_amd import flce
    s = make(M, 200, 264, 9)
    clean = flce.linear_forward(s["X"], s["W"], s["b"], "gelu")
    X = s["X"].clone()
    X[M // 2, 5] = float("nan")
    y = flce.linear_forward(X, s["W"], s["b"], "gelu")
    rest = torch.arange(M, device="cuda") != M // 2
    assert torch.isnan(y[M // 2]).all() and torch.equal(y[rest], clean[rest])
    W = s["W"].clone()
    W[11, 7] = float("nan")
    y = flce.linear_forward(s["X"], W, s["b"], "relu")
    cols = torch.arange(200, device="cuda") != 11
    assert torch.isnan(y[:, 11]).all() and torch.isfinite(y[:, cols]).all()
    # a NaN in pre or dy reaches what it should, of each act
    for act in ACTS[1:]:
        pre = torch.zeros(M, 200, device="cuda").bfloat16()
        pre[0, 3] = float("nan")
        dX, dW, db = flce.linear_backward(s["dy"], s["X"], s["W"], pre, act, bias_dtype=torch.float32)
        assert torch.isnan(dX[0]).all() and torch.isfinite(dX[1:]).all()
        assert torch.isnan(db[3]) and torch.isnan(dW[3]).all() and torch.isfinite(dW[4:]).all()


@pytest.mark.parametrize("M", [3, 33, 200])
@pytest.mark.parametrize("N,pad", [(64, 8), (100, 4), (131, 3)])
def test_strides_in_place_and_surroundings(M, N, pad):
    """Row strides of every matrix, results in the residual's place, what lies between rows left."""
    import torch
    from log_prob_amd import flce
    K = 136
    s = make(M, N, K, 12, residual="bf16")
    want, pre = flce.linear_forward(s["X"], s["W"], s["b"], "silu", s["r"], keep_pre=True)
    dy = s["dy"].bfloat16()
    grads = flce.linear_backward(dy, s["X"], s["W"], pre, "silu", bias_dtype=torch.float32)

    def wide(t, pad, fill=7.0):
        buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
        buf[:, :t.shape[1]] = t
        return buf, buf[:, :t.shape[1]]

    (_, X), (_, W) = wide(s["X"], 16, float("nan")), wide(s["W"], 8, float("nan"))
    for in_place in (False, True):
        rbuf, r = wide(s["r"], pad)
        obuf, o = (rbuf, r) if in_place else wide(torch.zeros_like(want), pad)
        pbuf, p = wide(torch.zeros_like(pre), pad)
        flce.linear_forward(X, W, s["b"], "silu", r, keep_pre=True, out=(o, p))
        assert torch.equal(o, want) and torch.equal(p, pre)
        assert (obuf[:, N:] == 7).all() and (pbuf[:, N:] == 7).all()
    _, d = wide(dy, pad, float("nan"))
    _, p = wide(pre, pad, float("nan"))
    xbuf, dX = wide(torch.zeros_like(s["X"]), pad)
    wbuf, dW = wide(torch.zeros_like(s["W"]), pad)
    db = torch.empty(N, device="cuda")
    flce.linear_backward(d, X, W, p, "silu", bias_dtype=torch.float32, out=(dX, dW, db))
    for a, b in zip((dX, dW, db), grads):
        assert torch.equal(a, b)
    assert (xbuf[:, K:] == 7).all() and (wbuf[:, K:] == 7).all()


def test_workspace_garbage_and_repeatability():
    """Split products and padded columns from a workspace of NaNs; results bitwise the same."""
    import torch
    from log_prob_amd import flce
    for M, N, K in ((16, 96, 4096), (40, 77, 2048), (600, 50, 64)):
        s = make(M, N, K, 13)
        fw, bw = flce.linear_workspace(M, N, K)
        nan = lambda n: torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
        want = flce.linear_forward(s["X"], s["W"], s["b"])
        assert torch.equal(flce.linear_forward(s["X"], s["W"], s["b"], workspace=nan(fw)), want)
        want = flce.linear_backward(s["dy"], s["X"], s["W"], bias_dtype=torch.float32)
        got = flce.linear_backward(s["dy"], s["X"], s["W"], bias_dtype=torch.float32, workspace=nan(bw))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_is_not_needed_and_empty_batches():
    import torch
    from log_prob_amd import flce
    s = make(20, 48, 64, 14)
    full = flce.linear_backward(s["dy"], s["X"], s["W"], bias_dtype=torch.bfloat16)
    for k in range(3):
        got = flce.linear_backward(s["dy"], s["X"], s["W"], need_dx=k == 0, need_dw=k == 1,
                                   bias_dtype=torch.bfloat16 if k == 2 else None)
        assert [g is not None for g in got] == [i == k for i in range(3)] and torch.equal(got[k], full[k])
    e = {k: v[:0] for k, v in s.items() if k in ("X", "dy")}
    assert flce.linear_forward(e["X"], s["W"], s["b"], "gelu").shape == (0, 48)
    dX, dW, db = flce.linear_backward(e["dy"], e["X"], s["W"], bias_dtype=torch.float32)
    assert dX.shape == (0, 64) and torch.equal(dW, torch.zeros_like(s["W"])) and torch.equal(db, torch.zeros(48, device="cuda"))


def test_refusals():
    import torch
    from log_prob_amd import flce
    s = make(12, 48, 64, 15, residual="bf16")
    X, W, b, r, dy = (s[k] for k in ("X", "W", "b", "r", "dy"))
    for call in (lambda: flce.linear_forward(X.float(), W), lambda: flce.linear_forward(X, W.float()),
                 lambda: flce.linear_forward(X, W, b.double()), lambda: flce.linear_forward(X, W, residual=r.half()),
                 lambda: flce.linear_forward(X, W, out_dtype=torch.float16),
                 lambda: flce.linear_backward(dy.half(), X, W),
                 lambda: flce.linear_backward(dy, X, W, bias_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: flce.linear_forward(X[0], W), lambda: flce.linear_forward(X, W[:, :32]),
                 lambda: flce.linear_forward(X.t(), W), lambda: flce.linear_forward(X, W, b[:5]),
                 lambda: flce.linear_forward(X, W, residual=r[:5]), lambda: flce.linear_forward(X, W, activation="tanh"),
                 lambda: flce.linear_forward(X, W.cpu()), lambda: flce.linear_backward(dy[:5], X, W),
                 lambda: flce.linear_backward(dy, X, W[:40]), lambda: flce.linear_backward(dy, X, W, activation="gelu"),
                 lambda: flce.linear_forward(X, W, out=torch.empty(12, 40, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: flce.linear_forward(X[:, :60].contiguous(), W[:, :60].contiguous()),   # K of 60
                 lambda: flce.linear_forward(X[:, 4:12], W[:, :8]),                             # rows not 16-byte aligned
                 lambda: flce.linear_forward(X, W, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda")[1:])
                 if flce.linear_workspace(12, 48, 64)[0] else flce.linear_forward(X[:, 4:12], W[:, :8])):
        with pytest.raises(flce.FlceError):
            call()
