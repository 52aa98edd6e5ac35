"""dX of up to 1024 values: formed from dpre before its rounding to bf16, whatever the number of rows."""
import numpy as np
import pytest

from tests import block_util as bu
from tests import ops_util as ou
from tests.test_linear_gpu import f64, make

pytestmark = pytest.mark.gpu

# (M, N, K), M K <= 1024: one row to 128; N of one share, a ragged one and many
SHAPES = [(1, 37832, 104), (1, 130, 1024), (2, 50257, 512), (4, 777, 256), (5, 3000, 200), (6, 1, 136), (10, 20001, 96),
          (16, 50257, 64), (33, 700, 24), (64, 64, 16), (127, 4099, 8), (128, 129, 8)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", None])
def test_values(M, N, K, act):
    """To the bounds of an fp32 dpre; and the norm of the error is that of one rounding to bf16 (1.66e-3 of
    the result's on average: uniform in half a step of 2^-8 2^e over values of 2^e to 2^(e + 1)), not of two
    (2.35e-3).  It varies by 1 / sqrt(2 n) of itself over n values: 2e-3 is 6 and 5 times that away for 500."""
    import torch
    from log_prob_amd import flce
    s = make(M, N, K, M + N + K, bias=None)
    pre = None if act is None else (s["dy"].flip(0) * 1.5).bfloat16()
    for dy in (s["dy"], s["dy"].bfloat16()):
        dX, dW, db = flce.linear_backward(dy, s["X"], s["W"], pre, act, bias_dtype=torch.float32)
        (want, bound), (dw, ew), (wb, eb) = bu.linear_grad_bounds(f64(dy), f64(s["X"]), f64(s["W"]), f64(pre), act, False)
        label = f"{M}x{N}x{K} {act} {dy.dtype}"
        ou.check_within(f64(dX), want, bound, label + " dX")
        if M * K >= 500 and N > 1:
            assert np.linalg.norm(f64(dX) - want) < 2e-3 * np.linalg.norm(want), label
        # the others as ever
        dw, ew = bu.linear_grad_bounds(f64(dy), f64(s["X"]), f64(s["W"]), f64(pre), act, True)[1]
        ou.check_within(f64(dW), dw, ew, label + " dW")
        ou.check_within(f64(db), wb, ou.half_step(torch.float32) * (np.abs(wb) + eb) + eb, label + " dbias")
        # alone, and into rows of another stride
        buf = torch.full((M, K + 5), 7.0, device="cuda").bfloat16()
        flce.linear_backward(dy, s["X"], s["W"], pre, act, need_dw=False, out=(buf[:, :K], None, None))
        assert torch.equal(buf[:, :K], dX) and (buf[:, K:] == 7).all()


@pytest.mark.parametrize("M,K", [(1, 8), (1, 1024), (3, 336), (4, 256), (5, 200), (17, 56), (128, 8)])
def test_what_a_rounding_would_lose(M, K):
    """1 + a 2^-12 against -1: bf16 has neither, the difference is exact in fp32."""
    import torch
    from log_prob_amd import flce
    N = 3000
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    a = torch.zeros(M, N // 2, device="cuda")
    a[:, :250] = torch.randint(-1, 2, (M, 250), generator=gen, device="cuda").float()
    dy = torch.ones(M, N, device="cuda")
    dy[:, ::2] += a.flip(1) * 2.0 ** -12
    W = torch.ones(N, K, device="cuda")
    W[1::2] = -1
    W[:, 1::2] *= 2
    dX = flce.linear_backward(dy, torch.zeros(M, K, device="cuda").bfloat16(), W.bfloat16(), need_dw=False)[0]
    want = (a.sum(1, keepdim=True) * 2.0 ** -12).expand(M, K).clone()
    want[:, 1::2] *= 2
    assert torch.equal(dX.float(), want) and want.any()
