"""Refusals of the residual block's calls and of log-probs from logits: all of them on the host,
before any HIP call, so no device is needed (pointers are never followed)."""
import pytest

from log_prob_amd import flce

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3
P = 1 << 20   # an address that is only looked at


def status(name, a):
    return getattr(flce.load(), name)(*a.values(), None)


def dropout(**kw):
    a = dict(x=P, xd=0, ldx=64, r=P, rd=0, ldr=64, M=4, H=64, p=0.1, seed=1, at=None, offset=0, y=P, yd=0, ldy=64)
    a.update(kw)
    return status("flce_dropout", a)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(H=0)), (UNSUPPORTED, dict(M=(1 << 30) + 1)),
    (UNSUPPORTED, dict(H=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21, ldr=1 << 21)),
    (INVALID, dict(xd=2)), (INVALID, dict(yd=-1)), (INVALID, dict(rd=5)),
    (INVALID, dict(p=-0.1)), (INVALID, dict(p=1.0001)), (INVALID, dict(p=float("nan"))),
    (UNSUPPORTED, dict(at=P + 4)), (INVALID, dict(x=None)), (INVALID, dict(y=None)),
    (INVALID, dict(ldx=63)), (INVALID, dict(ldr=0)), (INVALID, dict(ldy=8)),
    (UNSUPPORTED, dict(ldx=(1 << 40) + 1)), (UNSUPPORTED, dict(x=P + 1)), (UNSUPPORTED, dict(yd=1, y=P + 2)),
    (UNSUPPORTED, dict(rd=1, r=P + 2)),
])
def test_dropout(want, kw):
    assert dropout(**kw) == want
    assert flce.load().flce_last_error_message()


def forward(**kw):
    a = dict(X=P, ldx=64, W=P, ldw=64, b=P, bd=0, act=1, r=P, rd=0, ldr=32, M=40, N=32, K=64, out=P, od=0, ldo=32,
             pre=P, ldp=32, ws=P, wsb=1 << 30)
    a.update(kw)
    return status("flce_linear_forward", a)


SHAPES = [(INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=-8)), (UNSUPPORTED, dict(K=60)),
          (UNSUPPORTED, dict(M=(1 << 30) + 1)), (UNSUPPORTED, dict(N=(1 << 20) + 1)),
          (UNSUPPORTED, dict(K=(1 << 20) + 8)), (INVALID, dict(act=5)), (INVALID, dict(act=-1)),
          (INVALID, dict(bd=2)), (INVALID, dict(ldx=56)), (INVALID, dict(ldw=0)), (UNSUPPORTED, dict(ldx=65)),
          (UNSUPPORTED, dict(ldw=(1 << 21) + 8)), (UNSUPPORTED, dict(X=P + 8)), (UNSUPPORTED, dict(W=P + 2)),
          (INVALID, dict(X=None)), (INVALID, dict(W=None)), (UNSUPPORTED, dict(b=P + 1)),
          (INVALID, dict(ldp=31)), (UNSUPPORTED, dict(pre=P + 1)), (UNSUPPORTED, dict(ws=P + 128))]


@pytest.mark.parametrize("want,kw", SHAPES[:-1] + [
    (INVALID, dict(out=None)), (INVALID, dict(od=3)), (INVALID, dict(rd=3)), (INVALID, dict(ldo=31)),
    (INVALID, dict(ldr=31)), (UNSUPPORTED, dict(out=P + 1)), (UNSUPPORTED, dict(rd=1, r=P + 2)),
    # few tiles and a long K: the split's partial products need a workspace
    (TOO_SMALL, dict(K=4096, ldx=4096, ldw=4096, wsb=256)), (INVALID, dict(K=4096, ldx=4096, ldw=4096, ws=None)),
    (UNSUPPORTED, dict(K=4096, ldx=4096, ldw=4096, ws=P + 128)),
])
def test_linear_forward(want, kw):
    assert forward(**kw) == want
    assert flce.load().flce_last_error_message()


def backward(**kw):
    a = dict(dy=P, dyd=0, lddy=32, pre=P, ldp=32, act=1, X=P, ldx=64, W=P, ldw=64, M=40, N=32, K=64, dX=P, lddx=64,
             dW=P, lddw=64, b=P, bd=0, ws=P, wsb=1 << 30)
    a.update(kw)
    return status("flce_linear_backward", a)


@pytest.mark.parametrize("want,kw", SHAPES + [
    (INVALID, dict(dy=None)), (INVALID, dict(dyd=2)), (INVALID, dict(lddy=31)), (UNSUPPORTED, dict(dy=P + 1)),
    (INVALID, dict(pre=None)), (INVALID, dict(lddx=63)), (INVALID, dict(lddw=63)), (UNSUPPORTED, dict(dX=P + 1)),
    (UNSUPPORTED, dict(dW=P + 1)), (TOO_SMALL, dict(wsb=0)), (INVALID, dict(ws=None)),
])
def test_linear_backward(want, kw):
    assert backward(**kw) == want
    assert flce.load().flce_last_error_message()


def test_workspaces():
    assert flce.linear_workspace(1, 4096, 4096)[0] == 0 == flce.linear_workspace(16, 4096, 4096)[0]
    assert flce.linear_workspace(0, 16, 8)[0] == 0
    assert flce.linear_workspace(8192, 8192, 8192)[0] == 0
    assert flce.linear_workspace(64, 4096, 4096)[0] > 0
    assert flce.linear_workspace(5, 33, 64)[1] >= 5 * 40 * 2 + 33 * 4
    assert flce.token_logprobs_workspace(0, 1000, 5) == 0 == flce.token_logprobs_workspace(4096, 128256, 20)
    assert flce.token_logprobs_workspace(1, 128256, 5) > 0
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 12)):
        with pytest.raises(flce.FlceError):
            flce.linear_workspace(*bad)
    for bad in ((-1, 8, 0), (1, 0, 0), (1, 8, 9), (1, 1000, 129)):
        with pytest.raises(flce.FlceError):
            flce.token_logprobs_workspace(*bad)


def logprobs(**kw):
    a = dict(x=P, d=0, ldl=500, M=4096, V=500, t=P, n=2, ig=-100, s=1.0, k=3, lp=P, lse=P, ent=P, st=P, ids=P, tlp=P,
             ws=None, wsb=0)
    a.update(kw)
    return status("flce_token_logprobs", a)


def logprobs_grad(**kw):
    a = dict(x=P, d=0, ldl=500, M=4096, V=500, t=P, n=2, ig=-100, s=1.0, st=P, ent=P, ids=P, k=3, g=P, gt=P, ge=P,
             gl=P, dx=P, ldd=500)
    a.update(kw)
    return status("flce_token_logprobs_backward", a)


BOTH = [(INVALID, dict(M=-1)), (INVALID, dict(V=0)), (UNSUPPORTED, dict(V=(1 << 30) + 1, ldl=1 << 31)),
        (UNSUPPORTED, dict(M=(1 << 30) + 1)), (INVALID, dict(n=-1)), (INVALID, dict(k=-1)),
        (UNSUPPORTED, dict(n=1025)), (UNSUPPORTED, dict(k=129)), (INVALID, dict(V=2, k=3)),
        (INVALID, dict(s=0.0)), (INVALID, dict(s=-1.0)), (INVALID, dict(s=float("nan"))),
        (INVALID, dict(s=float("inf"))), (INVALID, dict(d=2)), (INVALID, dict(x=None)), (INVALID, dict(ldl=499)),
        (UNSUPPORTED, dict(x=P + 1)), (UNSUPPORTED, dict(t=P + 4)), (UNSUPPORTED, dict(ids=P + 4)),
        (UNSUPPORTED, dict(st=P + 2)), (INVALID, dict(t=None)), (INVALID, dict(st=None)), (INVALID, dict(ids=None))]


@pytest.mark.parametrize("want,kw", BOTH + [
    (INVALID, dict(lp=None)), (INVALID, dict(lse=None)), (INVALID, dict(tlp=None)), (UNSUPPORTED, dict(ent=P + 2)),
    (INVALID, dict(M=1, V=100000, ldl=100000)), (TOO_SMALL, dict(M=1, V=100000, ldl=100000, ws=P, wsb=64)),
    (UNSUPPORTED, dict(M=1, V=100000, ldl=100000, ws=P + 8, wsb=1 << 20))])
def test_token_logprobs(want, kw):
    assert logprobs(**kw) == want
    assert flce.load().flce_last_error_message()


@pytest.mark.parametrize("want,kw", BOTH + [
    (INVALID, dict(dx=None)), (INVALID, dict(ldd=10)), (INVALID, dict(ent=None)), (UNSUPPORTED, dict(g=P + 2)),
    (UNSUPPORTED, dict(gl=P + 1)), (INVALID, dict(ldl=600))])
def test_token_logprobs_backward(want, kw):
    # (the last: in place with another row stride)
    assert logprobs_grad(**kw) == want
    assert flce.load().flce_last_error_message()


def test_empty_calls_touch_nothing():
    assert dropout(M=0, x=None, y=None, r=None) == 0
    assert forward(M=0, X=None, W=None, b=None, r=None, out=None, pre=None, ws=None, wsb=0) == 0
    assert logprobs(M=0, x=None, t=None, lp=None, lse=None, ent=None, st=None, ids=None, tlp=None) == 0
    assert logprobs_grad(M=0, x=None, t=None, st=None, ent=None, ids=None, g=None, gt=None, ge=None, dx=None) == 0


def test_host_tensors_are_refused():
    import torch
    x, X = torch.zeros(2, 32), torch.zeros(2, 32, dtype=torch.bfloat16)
    t = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: flce.dropout(x, 0.1, 1), lambda: flce.dropout_backward(x, 0.1, 1),
                 lambda: flce.linear_forward(X, X), lambda: flce.linear_backward(X, X, X),
                 lambda: flce.token_logprobs(x, t), lambda: flce.token_logprobs_backward(x, t, x)):
        with pytest.raises(ValueError, match="expected a GPU tensor"):
            call()
    with pytest.raises(ValueError, match="activation"):
        flce.linear_forward(X, X, activation="tanh")
    for bad in (-1, 1 << 64):
        with pytest.raises(ValueError):
            flce._uint64(bad, "seed")
