"""Results in an input's place: refused where rows or elements would lie elsewhere (a thread would write
what another has yet to read), taken for a single row of any stride.  On the host, before any HIP call."""
import pytest

from log_prob_amd import flce
from tests.test_block_abi import INVALID, P, TOO_SMALL, dropout, forward, logprobs_grad

Q = P + 4096


@pytest.mark.parametrize("kw", [
    dict(r=None, ldy=72), dict(r=None, ldx=72), dict(r=Q, yd=1),        # y over x
    dict(x=Q, ldy=72), dict(x=Q, ldr=72), dict(x=Q, yd=1), dict(x=Q, rd=1),   # y over residual
    dict(x=Q, yd=1, M=1),
])
def test_dropout(kw):
    assert dropout(**kw) == INVALID
    assert b"place" in flce.load().flce_last_error_message()


@pytest.mark.parametrize("kw", [dict(ldo=40), dict(ldr=40), dict(od=1), dict(rd=1), dict(rd=1, M=1)])
def test_linear(kw):
    assert forward(**kw) == INVALID
    assert b"place" in flce.load().flce_last_error_message()


def test_what_agrees_or_has_one_row_is_taken():
    # (as far as the workspace, which a long K needs)
    long = dict(K=4096, ldx=4096, ldw=4096, wsb=256, pre=None)
    assert forward(**long) == TOO_SMALL
    assert forward(**long, ldr=40, ldo=40) == TOO_SMALL
    assert forward(**long, r=Q, ldr=40, rd=1) == TOO_SMALL


def test_log_prob_gradient():
    assert logprobs_grad(ldl=600) == INVALID
    # a single row's stride means nothing: the call gets as far as what follows
    assert logprobs_grad(M=1, ldl=600, st=None) == INVALID
    assert b"stats is NULL" in flce.load().flce_last_error_message()
