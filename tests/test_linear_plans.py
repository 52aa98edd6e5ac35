"""Which kernel a few rows take, seen by the workspace: W streamed needs none, tiles that split K do."""
import pytest

from log_prob_amd import flce

STREAMED = [(3, 512, 8192), (16, 512, 8192), (16, 1024, 8192), (3, 2048, 8192), (16, 4096, 4096), (32, 4096, 4096)]


@pytest.mark.parametrize("M,N,K", STREAMED)
def test_streamed(M, N, K):
    assert flce.linear_workspace(M, N, K)[0] == 0


def test_tiles():
    assert flce.linear_workspace(32, 2048, 8192)[0] > 0 and flce.linear_workspace(33, 1024, 8192)[0] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", STREAMED[:4])
def test_values(M, N, K):
    from tests.test_linear_gpu import check_forward, make
    check_forward(make(M, N, K, M + N, bias="fp32", residual="bf16"), "silu", "bf16", f"{M}x{N}x{K}")
