"""The fp64 definitions of the residual block and of log-probs from logits: known answers,
differences, torch in float64."""
import numpy as np
import pytest

from oracle import block_ref as ref

ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("counter,key,want", [
    # the known-answer vectors published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(ref.philox(counter, key)) == want


def test_dropout_keeps_what_it_should():
    x = np.random.default_rng(1).normal(size=(64, 203))
    for p in (0.0, 0.1, 0.5, 1.0):
        if p == 1.0:
            assert (ref.dropout_bits(4, 16, 1, 2) < 65536).all()
            continue
        y = ref.dropout(x, p, 5, 7, residual=x)
        kept = y != x
        n = x.size
        assert abs(kept.mean() - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n) + 1e-9
        q = round(65536 * p) / 65536
        np.testing.assert_allclose(y[kept], (x + x / (1 - q))[kept])
    a, b = ref.dropout_bits(8, 64, 5, 7), ref.dropout_bits(8, 64, 5, 8)
    assert (a != b).mean() > 0.99 and np.array_equal(a[:, :21], ref.dropout_bits(8, 21, 5, 7))


@pytest.mark.parametrize("name", ACTS)
def test_activations_against_torch(name):
    import torch
    import torch.nn.functional as F
    z = torch.linspace(-9, 9, 401, dtype=torch.float64, requires_grad=True)
    f = {None: lambda v: v, "relu": F.relu, "gelu": F.gelu,
         "gelu_tanh": lambda v: F.gelu(v, approximate="tanh"), "silu": F.silu}[name]
    y = f(z)
    (g,) = torch.autograd.grad(y.sum(), z)
    np.testing.assert_allclose(ref.act(z.detach().numpy(), name), y.detach().numpy(), atol=1e-12)
    want = g.numpy().copy()
    if name == "relu":
        want[z.detach().numpy() == 0] = 0.0
    np.testing.assert_allclose(ref.act_slope(z.detach().numpy(), name), want, atol=1e-12)


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradient_by_differences(name):
    r = np.random.default_rng(3)
    X, W, b, c = r.normal(size=(5, 8)), r.normal(size=(6, 8)), r.normal(size=6), r.normal(size=(5, 6))
    loss = lambda X, W, b: (c * ref.linear(X, W, b, name, X[:, :6])[0]).sum()
    pre = ref.linear(X, W, b, name, None)[1]
    dX, dW, db, _ = ref.linear_grad(c, X, W, pre, name)
    dX = dX + np.pad(c, ((0, 0), (0, 2)))   # the residual's share
    h = 1e-6
    for k, (a, g) in enumerate(((X, dX), (W, dW), (b, db))):
        for i in np.ndindex(a.shape):
            args = [X.copy(), W.copy(), b.copy()]
            args[k][i] += h
            up = loss(*args)
            args[k][i] -= 2 * h
            assert abs((up - loss(*args)) / (2 * h) - g[i]) <= 1e-6 * (1 + abs(g[i]))


def test_logprobs_against_torch():
    import torch
    r = np.random.default_rng(4)
    x = r.normal(size=(7, 33)) * 3
    x[2, :20] = -np.inf
    t = r.integers(0, 33, size=(7, 4))
    t[1, 2], t[3, 0], t[4, 1] = -100, 33, -1
    z = torch.tensor(x, requires_grad=True)
    lp = torch.log_softmax(0.7 * z, 1)
    ent = -(torch.exp(lp) * torch.where(torch.isinf(lp), 0.0, lp)).sum(1)
    o = ref.token_logprobs(x, t, -100, 0.7, 5)
    ok = ref.valid_tokens(t, 33, -100)
    want = lp.detach().gather(1, torch.tensor(np.where(ok, t, 0))).numpy()
    np.testing.assert_allclose(o["logprob"], np.where(ok, want, 0.0), atol=1e-12)
    np.testing.assert_allclose(o["lse"], torch.logsumexp(0.7 * z, 1).detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(o["entropy"], ent.detach().numpy(), atol=1e-12)
    top = torch.topk(z.detach(), 5, dim=1)
    assert np.array_equal(o["top_ids"], top.indices.numpy())
    np.testing.assert_allclose(o["top_logprob"], lp.detach().gather(1, top.indices).numpy(), atol=1e-12)
    np.testing.assert_allclose(o["stats"][:, 0] * 0.7 + o["stats"][:, 1], o["lse"], atol=1e-12)


def test_logprob_gradient_by_differences():
    r = np.random.default_rng(5)
    x = r.normal(size=(4, 9))
    x[1, 3] = -np.inf
    t = r.integers(0, 9, size=(4, 3))
    t[0, 0], t[2] = -100, 5     # an ignored token; one token three times
    t[t == 3] = 4
    g, gt, ge, gl = r.normal(size=(4, 3)), r.normal(size=(4, 2)), r.normal(size=4), r.normal(size=4)
    ids = ref.token_logprobs(x, t, n_top=2)["top_ids"]

    def loss(x):
        o = ref.token_logprobs(x, t, -100, 1.3)
        own = np.take_along_axis(ref._rows(x, 1.3)[0], ids, 1)
        return (o["logprob"] * g).sum() + (own * gt).sum() + (o["entropy"] * ge).sum() + (o["lse"] * gl).sum()

    d = ref.token_logprobs_grad(x, t, g, -100, 1.3, ids, gt, ge, gl)
    for i in np.ndindex(x.shape):
        if np.isinf(x[i]):
            assert d[i] == 0
            continue
        a, b = x.copy(), x.copy()
        a[i] += 1e-6
        b[i] -= 1e-6
        assert abs((loss(a) - loss(b)) / 2e-6 - d[i]) <= 1e-6


def test_odd_rows():
    x = np.array([[1.0, np.nan, 0.0, 2.0], [-np.inf] * 4, [np.inf, 0.0, np.inf, -1.0], [5.0, 5.0, -0.0, 0.0]])
    t = np.zeros((4, 1), np.int64)
    o = ref.token_logprobs(x, t, n_top=4)
    assert o["top_ids"].tolist() == [[3, 0, 2, 1], [0, 1, 2, 3], [0, 2, 1, 3], [0, 1, 2, 3]]
    assert np.isnan(o["logprob"][[0, 2], 0]).all() and o["logprob"][1, 0] == -np.inf
    assert o["lse"][1] == -np.inf and o["entropy"][1] == 0 and np.isnan(o["lse"][0])
