"""Layer norm forward and backward on the GPU against the fp64 definition, with bounds
counted from the roundings of the 32-bit path (tests/ops_util.py)."""
import numpy as np
import pytest

from oracle import ops_ref as ops
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

EPS = 1e-5
KINDS = [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")]


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def make(M, H, x, y, p, seed, offset=0.5):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    loud = torch.where(torch.rand(H, generator=gen, device="cuda") < 0.02, 12.0, 1.0)
    return dict(x=(n(M, H) * loud + offset * n(M, 1)).to(dt(x)), w=(1 + 0.1 * n(H)).to(dt(p)),
                b=(0.1 * n(H)).to(dt(p)), dy=n(M, H).to(dt(y)))


def check(s, y_dtype, label, weight=True, bias=True, eps=EPS):
    import torch
    from log_prob_amd import flce
    x, w, b, dy = s["x"], s["w"] if weight else None, s["b"] if bias else None, s["dy"]
    y, mean, rstd = flce.layer_norm_forward(x, w, b, eps, out_dtype=y_dtype)
    assert y.dtype == y_dtype and mean.dtype == rstd.dtype == torch.float32
    x64, w64, b64 = ou.np64(x), None if w is None else ou.np64(w), None if b is None else ou.np64(b)
    want = ops.layer_norm(x64, w64, b64, eps)
    bounds = ou.norm_forward_bounds(x64, w64, b64, eps, *want, ou.half_step(y_dtype))
    for name, got, ref, bound in zip(("y", "mean", "rstd"), (y, mean, rstd), want, bounds):
        ou.check_within(ou.np64(got), ref, bound, f"{label} {name}")
    dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.dtype == x.dtype
    m64, r64, dy64 = ou.np64(mean), ou.np64(rstd), ou.np64(dy)
    want = ops.layer_norm_grad(dy64, x64, m64, r64, w64)
    bounds = ou.norm_backward_bounds(dy64, x64, m64, r64, w64, *want, ou.half_step(x.dtype),
                                     ou.half_step(dw.dtype))
    for name, got, ref, bound in zip(("dx", "dweight", "dbias"), (dx, dw, db), want, bounds):
        ou.check_within(ou.np64(got), ref, bound, f"{label} {name}")
    return y, mean, rstd, dx, dw, db


# one element to many; whole chunks and odd lengths; every row layout's first and last width
SHAPES = [(1, 1), (3, 2), (1, 8), (5, 7), (2, 40), (65, 64), (33, 136), (7, 511), (9, 512),
          (4, 513), (6, 520), (5, 1000), (3, 1024), (4, 1025), (7, 1032), (3, 2047), (2, 2048),
          (5, 2056), (1, 4096), (3, 4099), (2, 4104), (2, 8191), (3, 8192), (1, 8200), (2, 10007),
          (3, 16384), (2, 16392), (1, 20001)]


@pytest.mark.parametrize("x,y", KINDS)
@pytest.mark.parametrize("M,H", SHAPES)
def test_shapes(M, H, x, y):
    for p in {"fp32", y}:
        check(make(M, H, x, y, p, 1000 * M + H), dt(y), f"{M}x{H} {x}->{y} {p}")


@pytest.mark.parametrize("M,H,x,y", [(4097, 136, "bf16", "bf16"), (1025, 1000, "fp32", "fp32"),
                                     (2500, 2048, "bf16", "bf16"), (1100, 4096, "fp32", "bf16"),
                                     (700, 8192, "bf16", "bf16"), (300, 8200, "fp32", "fp32"),
                                     (600, 20000, "bf16", "bf16"), (5000, 33, "bf16", "bf16")])
def test_many_rows(M, H, x, y):
    """More rows than one pass of the workgroups covers."""
    check(make(M, H, x, y, "fp32", 7), dt(y), f"{M}x{H}")


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_without_parameters(weight, bias):
    check(make(9, 200, "bf16", "bf16", "bf16", 3), dt("bf16"), "no params", weight, bias)


def test_large_offset_keeps_its_digits():
    """A row offset far above the spread: the centred second pass carries the variance."""
    s = make(6, 2048, "fp32", "fp32", "fp32", 5)
    s["x"] = s["x"] * 0.01 + 1000.0
    check(s, dt("fp32"), "offset")


def test_constant_rows():
    """No spread at all: rstd = eps^-1/2, y = bias, and the gradient is finite."""
    import torch
    s = make(4, 264, "fp32", "fp32", "fp32", 6)
    s["x"] = torch.full_like(s["x"], 3.0)
    y, mean, rstd, dx, dw, db = check(s, dt("fp32"), "constant")
    assert torch.equal(y, s["b"].expand_as(y)) and torch.equal(dw, torch.zeros_like(dw))


def test_nonfinite_rows_stay_in_their_rows():
    import torch
    from log_prob_amd import flce
    s = make(8, 1000, "bf16", "bf16", "bf16", 8)
    clean = flce.layer_norm_forward(s["x"], s["w"], s["b"], EPS)
    x = s["x"].clone()
    x[2, 5] = float("nan")
    x[6, 999] = float("inf")
    y, mean, rstd = flce.layer_norm_forward(x, s["w"], s["b"], EPS)
    keep = torch.tensor([0, 1, 3, 4, 5, 7], device="cuda")
    assert torch.isnan(y[2]).all() and torch.isnan(y[6]).any()
    assert torch.isnan(mean[2]) and torch.isnan(rstd[2]) and torch.isnan(rstd[6])
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(mean[keep], clean[1][keep])


@pytest.mark.parametrize("H", [264, 2048, 4104, 9000])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (16, 8)])
def test_row_strides(H, pad, shift):
    """Rows inside wider rows, at addresses that are and are not multiples of 16 bytes; what
    lies between the rows is left as it was."""
    import torch
    from log_prob_amd import flce
    M = 5
    s = make(M, H, "bf16", "bf16", "bf16", 9)
    ref = check(s, torch.bfloat16, "contiguous")

    def wide(t, fill):
        buf = torch.full((M * (H + pad) + shift,), fill, dtype=t.dtype, device="cuda")
        view = buf[shift:].view(M, H + pad)[:, :H]
        view.copy_(t)
        return buf, view

    _, x = wide(s["x"], 1.0)
    _, dy = wide(s["dy"], 1.0)
    ybuf, y = wide(torch.zeros_like(s["x"]), 7.0)
    dbuf, dx = wide(torch.zeros_like(s["x"]), 7.0)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    flce.layer_norm_forward(x, s["w"], s["b"], EPS, out=(y, mean, rstd))
    dw, db = torch.empty_like(s["w"]), torch.empty_like(s["w"])
    flce.layer_norm_backward(dy, x, mean, rstd, s["w"], out=(dx, dw, db))
    for name, a, b in zip(("y", "mean", "rstd", "dx", "dw", "db"), (y, mean, rstd, dx, dw, db), ref):
        assert torch.equal(a, b), name
    for buf in (ybuf, dbuf):
        gaps = buf[shift:].view(M, H + pad)[:, H:]
        assert (gaps == 7.0).all() and (buf[:shift] == 7.0).all()


def test_in_place():
    import torch
    from log_prob_amd import flce
    for H in (1000, 17000):
        s = make(6, H, "bf16", "bf16", "bf16", 10)
        y, mean, rstd, dx, dw, db = check(s, torch.bfloat16, "apart")
        x, dy = s["x"].clone(), s["dy"].clone()
        flce.layer_norm_forward(x, s["w"], s["b"], EPS, out=(x, mean, rstd))
        assert torch.equal(x, y)
        flce.layer_norm_backward(dy, s["x"], mean, rstd, s["w"], out=(dy, dw, db))
        assert torch.equal(dy, dx)


def test_no_rows():
    import torch
    from log_prob_amd import flce
    x = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(264, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = flce.layer_norm_forward(x, w, None, EPS)
    assert y.shape == (0, 264) and mean.shape == (0,)
    dx, dw, db = flce.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 264) and not dw.any() and not db.any()


def test_repeatable_and_parameters_optional():
    import torch
    from log_prob_amd import flce
    s = make(3000, 1000, "bf16", "bf16", "fp32", 12)
    y, mean, rstd = flce.layer_norm_forward(s["x"], s["w"], s["b"], EPS)
    first = flce.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["w"])
    ws = torch.full((flce.layer_norm_backward_workspace(3000, 1000) // 4,), float("nan"), device="cuda")
    again = flce.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["w"], workspace=ws)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    dx, dw, db = flce.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["w"], need_params=False)
    assert torch.equal(dx, first[0]) and dw is None and db is None


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("x,y", KINDS)
@pytest.mark.parametrize("M,H", [(1, 8), (5, 33), (3, 512), (513, 1000), (2, 2048), (300, 4104),
                                 (3, 8200), (2, 17001)])
def test_checkpoint(M, H, x, y, fmt):
    """The forward's 8-bit copy is the quantiser's, and the backward is that of its values."""
    import torch
    from log_prob_amd import flce
    s = make(M, H, x, y, "fp32", 31 * M + H)
    plain = flce.layer_norm_forward(s["x"], s["w"], s["b"], EPS, out_dtype=dt(y))
    *got, kept = flce.layer_norm_forward(s["x"], s["w"], s["b"], EPS, out_dtype=dt(y), checkpoint=fmt)
    for a, b in zip(got, plain):
        assert torch.equal(a, b)
    q = flce.mx_quantize(s["x"], fmt)
    assert torch.equal(q.codes, kept.codes) and torch.equal(q.scales, kept.scales)
    y_, mean, rstd = got
    v = ops.rounded(ou.np64(s["x"]), fmt)
    m64, r64, dy64, w64 = (ou.np64(t) for t in (mean, rstd, s["dy"], s["w"]))
    want = ops.layer_norm_grad(dy64, v, m64, r64, w64)
    for dx_dtype in {torch.float32, dt(y)}:
        dx, dw, db = flce.layer_norm_backward(s["dy"], kept, mean, rstd, s["w"], dx_dtype=dx_dtype)
        bounds = ou.norm_backward_bounds(dy64, v, m64, r64, w64, *want, ou.half_step(dx_dtype), ou.U32)
        for name, g, ref, bound in zip(("dx", "dweight", "dbias"), (dx, dw, db), want, bounds):
            ou.check_within(ou.np64(g), ref, bound, f"{fmt} {name}")
