"""Products of so many rows that small tiles would not fit a launch: larger ones are taken, and the
workspace query refuses what the call refuses.  On the host; the last test runs one."""
import ctypes

import pytest

from log_prob_amd import flce
from tests.test_block_abi import TOO_SMALL, UNSUPPORTED, backward, forward

TALL = [(1 << 30, 8, 8), (1 << 30, 256, 64), ((1 << 30) - 77, 100, 16), (1 << 29, 64, 64), (1 << 29, 512, 8),
        (300_000_000, 8, 1024)]
# half a terabyte and more of X or results, whatever the tile
TOO_TALL = [(1 << 30, 1 << 10, 8), (1 << 30, 8, 1 << 10), (1 << 28, 1 << 14, 64)]


def query(M, N, K, which):
    b = ctypes.c_size_t(12345)
    args = (ctypes.byref(b), None) if which == "forward" else (None, ctypes.byref(b))
    return flce.load().flce_linear_workspace(M, N, K, *args), b.value


@pytest.mark.parametrize("M,N,K", TALL)
def test_tall_products_are_taken(M, N, K):
    assert query(M, N, K, "forward") == (0, 0)
    st, need = query(M, N, K, "backward")
    assert st == 0 and need >= M * ((N + 7) // 8 * 8) * 2
    # the call gets as far as its workspace
    assert backward(M=M, N=N, K=K, lddy=N, ldp=N, ldx=K, ldw=K, lddx=K, lddw=K, wsb=0) == TOO_SMALL


@pytest.mark.parametrize("M,N,K", TOO_TALL)
def test_the_query_refuses_with_the_call(M, N, K):
    if N > 512:
        assert query(M, N, K, "forward")[0] == UNSUPPORTED
        assert forward(M=M, N=N, K=K, ldx=K, ldw=K, ldr=N, ldo=N, ldp=N) == UNSUPPORTED
    else:
        assert query(M, N, K, "backward")[0] == UNSUPPORTED
        assert backward(M=M, N=N, K=K, lddy=N, ldp=N, ldx=K, ldw=K, lddx=K, lddw=K) == UNSUPPORTED


@pytest.mark.gpu
def test_a_tall_product():
    """2^30 x 8 from a K of 8, and dX: rows at both ends as in a call of their own (68 GB)."""
    import gc
    import torch
    M, N, K, n = 1 << 30, 8, 8, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(N, K, generator=gen, device="cuda").bfloat16()
    X = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    X.view(1 << 10, 1 << 20, K).copy_(torch.randn(1 << 20, K, generator=gen, device="cuda"))
    X[-n:] *= 0.5
    y = flce.linear_forward(X, W, activation="relu")
    assert torch.equal(y[:n], flce.linear_forward(X[:n].clone(), W, activation="relu"))
    assert torch.equal(y[-n:], flce.linear_forward(X[-n:].clone(), W, activation="relu"))
    assert torch.equal(y[M // 2:M // 2 + n], y[:n])
    dX = flce.linear_backward(y, X, W, need_dw=False)[0]
    for s in (slice(0, n), slice(M - n, M)):
        assert torch.equal(dX[s], flce.linear_backward(y[s].clone(), X[s].clone(), W, need_dw=False)[0])
    del X, y, dX
    gc.collect()
    torch.cuda.empty_cache()
