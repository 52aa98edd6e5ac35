"""Calls around the head that the documentation allows at the ends of their ranges: the largest
and smallest block scales, gradients over their own input, bf16 parameters of fp32 rows, an
input changed before its backward."""
import numpy as np
import pytest

from oracle import ops_ref as ops
from tests import ops_util as ou
from tests.test_mx_head_gpu import forward_bounds

pytestmark = pytest.mark.gpu

EPS = 1e-5


# the product quantising its own tokens, few tokens, token tiles, tiles of 256 with merges of
# either kind
@pytest.mark.parametrize("M,V", [(1, 700), (8, 700), (40, 700), (140, 1300), (500, 32100), (1100, 40000)])
@pytest.mark.parametrize("up,down", [(125, -121), (120, -120), (-120, 120), (-124, 125)])
def test_scales_far_apart(M, V, up, down):
    """X near one end of bf16's range and W near the other: logits of ordinary size, from block
    scales whose product with either operand alone passes fp32's range."""
    import torch
    from log_prob_amd import flce
    H = 264
    gen = torch.Generator(device="cuda").manual_seed(M + 1)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    X = torch.ldexp(n(M, H), torch.tensor(up, device="cuda")).bfloat16()
    X[:, 40:72] = 0
    W = flce.mx_quantize(torch.ldexp(n(V, H) / H ** 0.5, torch.tensor(down, device="cuda")), "mxfp4")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    assert X.isfinite().all() and (X.abs().max() > 2.0 ** 118 or X.abs().max() < 2.0 ** -116)
    Wv = ou.np64(flce.mx_dequantize(W, torch.float32))
    Xv = ops.rounded(ou.np64(X), "mxfp4")
    z = Xv @ Wv.T
    e = (H + 2) * 2 * ou.U32 * (np.abs(Xv) @ np.abs(Wv).T)
    got = flce.mxfp4_logits(X, W, out_dtype=torch.float32)
    ou.check_within(ou.np64(got), z, ou.U32 * (np.abs(z) + e) + e, "logits")
    want = ops.fp4_forward(ou.np64(X), Wv, t.cpu().numpy())
    bounds = forward_bounds(z, e, V)
    for name, a, b in zip(("logprob", "lse", "entropy"), flce.mxfp4_forward(X, W, t), bounds):
        ou.check_within(ou.np64(a), want[name], b, name)


@pytest.mark.parametrize("H", [100, 1000, 1001, 4104, 8200, 17003])
@pytest.mark.parametrize("over", ["x", "dy"])
def test_gradient_over_its_input(H, over):
    import torch
    from log_prob_amd import flce
    gen = torch.Generator(device="cuda").manual_seed(H)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        x, dy, w = n(300, H).to(dtype), n(300, H).to(dtype), n(H)
        _, mean, rstd = flce.layer_norm_forward(x, w, None, EPS)
        dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w)
        x2, dy2 = x.clone(), dy.clone()
        dw2, db2 = torch.empty_like(w), torch.empty_like(w)
        out = x2 if over == "x" else dy2
        flce.layer_norm_backward(dy2, x2, mean, rstd, w, out=(out, dw2, db2))
        assert torch.equal(out, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("H", [33, 264, 2048, 17001])
def test_bf16_parameters_of_fp32_rows(H):
    import torch
    from log_prob_amd import flce
    gen = torch.Generator(device="cuda").manual_seed(H)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy, w, b = n(7, H), n(7, H), (1 + 0.1 * n(H)).bfloat16(), n(H).bfloat16()
    y, mean, rstd = flce.layer_norm_forward(x, w, b, EPS)
    x64, w64, b64 = ou.np64(x), ou.np64(w), ou.np64(b)
    want = ops.layer_norm(x64, w64, b64, EPS)
    for name, g, r, e in zip(("y", "mean", "rstd"), (y, mean, rstd), want,
                             ou.norm_forward_bounds(x64, w64, b64, EPS, *want, ou.U32)):
        ou.check_within(ou.np64(g), r, e, name)
    got = flce.layer_norm_backward(dy, x, mean, rstd, w)
    assert got[1].dtype == got[2].dtype == torch.bfloat16
    m64, r64, dy64 = ou.np64(mean), ou.np64(rstd), ou.np64(dy)
    want = ops.layer_norm_grad(dy64, x64, m64, r64, w64)
    for name, g, r, e in zip(("dx", "dw", "db"), got, want,
                             ou.norm_backward_bounds(dy64, x64, m64, r64, w64, *want, ou.U32, ou.U16)):
        ou.check_within(ou.np64(g), r, e, name)


def test_an_input_changed_before_its_backward_is_noticed():
    """The graph keeps x itself: torch refuses.  It keeps a copy in 8 bits: nothing to refuse."""
    import torch
    from log_prob_amd import autograd
    for shape in ((6, 64), (2, 3, 64)):
        x = torch.randn(shape, device="cuda")
        w = torch.ones(64, device="cuda", requires_grad=True)
        y = autograd.layer_norm(x, w, None)
        x.add_(1.0)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        y = autograd.layer_norm(x, w, None, checkpoint="mxfp8")
        x.add_(1.0)
        y.sum().backward()
