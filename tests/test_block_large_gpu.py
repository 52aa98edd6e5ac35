"""The residual block on matrices whose offsets pass 32 bits: last rows against the definitions, or
against the same rows in a call of their own."""
import numpy as np
import pytest

from oracle import block_ref as ref
from tests import block_util as bu
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    """These tests hold up to 40 GB: give back what is cached on both sides."""
    import gc
    import torch
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_dropout():
    """560000 x 8193 bf16: 4.6e9 elements."""
    import torch
    from log_prob_amd import flce
    M, H, n = 560000, 8193, 3
    x = torch.ones(M, H, dtype=torch.bfloat16, device="cuda")
    y = flce.dropout(x, 0.25, 77, 5, residual=x)
    got = y[-n:].float().cpu().numpy() > 1.5
    for i in range(n):
        for b in (0, 1, 511, 1023, 1024):
            words = ref.philox((b, M - n + i, 5, 0), (77, 0))
            bits = np.array([h for w in words for h in (w & 0xFFFF, w >> 16)])[: max(0, min(8, H - 8 * b))]
            assert np.array_equal(got[i, 8 * b:8 * b + 8], bits >= 16384), (i, b)
    y.copy_(x)
    flce.dropout(y, 0.25, 77, 5, residual=x, out=y)
    assert np.array_equal(y[-n:].float().cpu().numpy() > 1.5, got)


def test_linear():
    """90000 x 50256 results (4.5e9) from a K of 72, and back."""
    import torch
    from log_prob_amd import flce
    M, N, K, n = 90000, 50256, 72, 40
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(N, K, generator=gen, device="cuda") / 8).bfloat16()
    y, pre = flce.linear_forward(X, W, None, "silu", keep_pre=True)
    want, pre64, e, ep = bu.linear_bounds(ou.np64(X[-n:]), ou.np64(W), None, "silu", None, ou.U16)
    ou.check_within(ou.np64(y[-n:]), want, e, "out")
    ou.check_within(ou.np64(pre[-n:]), pre64, ep, "pre")
    # a gradient in the last rows alone: dX is theirs, dW what they leave
    y.zero_()
    y[-n:] = torch.randn(n, N, generator=gen, device="cuda")
    dX, dW, db = flce.linear_backward(y, X, W, pre, "silu", bias_dtype=torch.float32)
    (wx, ex), (ww, ew), (wb, eb) = bu.linear_grad_bounds(ou.np64(y[-n:]), ou.np64(X[-n:]), ou.np64(W), ou.np64(pre[-n:]),
                                                         "silu", True)
    ou.check_within(ou.np64(dX[-n:]), wx, ex, "dX")
    assert (dX[:-n] == 0).all()
    # (zeros join the sums without a rounding: the bounds of the rows alone hold)
    ou.check_within(ou.np64(dW), ww, ew, "dW")
    ou.check_within(ou.np64(db), wb, eb, "dbias")
