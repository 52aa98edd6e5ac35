"""The gradient of log-probs and entropy from logits at the largest scales and gradients that are
accepted, under masks: a logit without probability has no gradient, however large its factors are."""
import numpy as np
import pytest

from oracle import block_ref as ref
from tests import block_util as bu
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


def masked_logits(M, V, dtype, scale, seed):
    """scale * logits of a common spread, with -inf, the type's lowest value and -5 among them (at these
    scales far below every other); a row of -inf alone, one of the lowest value alone, one token alone."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = (3.0 / scale * torch.randn(M, V, generator=gen, device="cuda")).to(dtype)
    u = torch.rand(M, V, generator=gen, device="cuda")
    z[u < 0.2] = -float("inf")
    z[(u > 0.2) & (u < 0.3)] = torch.finfo(dtype).min
    z[(u > 0.3) & (u < 0.4)] = -5.0
    z[1], z[2], z[3, 1:] = -float("inf"), torch.finfo(dtype).min, -float("inf")
    t = torch.randint(0, V, (M, 3), generator=gen, device="cuda")
    t[0, 1], t[3, 0] = -100, 0
    return z, t


def check(z, t, scale, g, b, label):
    """dlogits against the definition, bounds as in tests/test_token_logprobs_gpu.py."""
    from log_prob_amd import flce
    M, V = z.shape
    r = flce.token_logprobs(z, t, -100, scale, 0, True)
    got = ou.np64(flce.token_logprobs_backward(z, t, r.stats, r.entropy, None, g, None, b, None, -100, scale))
    x, tn, gn = ou.np64(z), t.cpu().numpy(), ou.np64(g)
    bn = np.zeros(M) if b is None else np.abs(ou.np64(b))
    want = ref.token_logprobs_grad(x, tn, gn, -100, scale, None, None, None if b is None else ou.np64(b))
    logp, d, logs, *_ = ref._rows(x, scale)
    p = np.exp(np.where(np.isfinite(logp), logp, -np.inf))
    lp, ad = np.where(p > 0, np.abs(logp), 0), np.where(p > 0, np.abs(d), 0)
    # (nothing lies where fp32 has no e^d and 64 bits have one)
    assert (ad < 80).all()
    e_s, e_u = bu.sum_error(x, scale, V)
    ent = np.abs(ref.token_logprobs(x, tn, -100, scale)["entropy"])
    mag = np.abs(gn).sum(1)
    rel = 2.0 ** -20 + e_s[:, None] + 6 * ou.U32 * (lp + ad + np.abs(logs)[:, None])
    coef = mag[:, None] + bn[:, None] * (lp + ent[:, None])
    e = scale * p * (coef * rel + bn[:, None] * (rel + (e_s + e_u)[:, None]) + mag[:, None] * (3 + 8) * ou.U32)
    add = np.zeros((M, V))
    for m in range(M):
        for j in range(3):
            if tn[m, j] >= 0:
                add[m, tn[m, j]] += abs(gn[m, j])
    e = e + scale * add * (3 + 4) * ou.U32
    ou.check_within(got, want, ou.half_step(z.dtype) * (np.abs(want) + e) + e, label)
    assert (got[(p == 0) & (add == 0)] == 0).all(), label


@pytest.mark.parametrize("V", [70, 9001])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1.0, 1e9, 1e18, 2.0 ** 64])
def test_large_scales(scale, x, V):
    import torch
    scale = float(np.float32(scale))
    z, t = masked_logits(6, V, {"bf16": torch.bfloat16, "fp32": torch.float32}[x], scale, V)
    gen = torch.Generator(device="cuda").manual_seed(2)
    g, b = torch.randn(6, 3, generator=gen, device="cuda"), torch.randn(6, generator=gen, device="cuda")
    check(z, t, scale, g, b, f"{scale} {x} both")
    check(z, t, scale, g, None, f"{scale} {x} log-probs")


@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("scale,b", [(1.0, 4e8), (1.0, 1e36), (0.5, -1e30), (1e9, 1e9), (2.0 ** 64, 4e18)])
def test_large_gradients_of_the_entropy(scale, b, x):
    import torch
    scale = float(np.float32(scale))
    z, t = masked_logits(5, 2100, {"bf16": torch.bfloat16, "fp32": torch.float32}[x], scale, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = torch.randn(5, 3, generator=gen, device="cuda")
    check(z, t, scale, g, torch.full((5,), b, device="cuda"), f"{scale} {b} {x}")


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 64])
def test_nan_still_reaches_its_row(scale):
    import torch
    from log_prob_amd import flce
    z, t = masked_logits(5, 300, torch.float32, scale, 5)
    z[0, 7], z[4, 9] = float("nan"), float("inf")
    r = flce.token_logprobs(z, t, -100, scale, 0, True)
    d = flce.token_logprobs_backward(z, t, r.stats, r.entropy, None, torch.ones(5, 3, device="cuda"), None,
                                     torch.ones(5, device="cuda"), None, -100, scale)
    assert torch.isnan(d[0]).all() and torch.isnan(d[4]).all() and torch.isfinite(d[1:4]).all()


@pytest.mark.parametrize("which", ["logprob", "entropy", "lse"])
def test_nan_gradients_reach_masked_logits_too(which):
    import torch
    from log_prob_amd import flce
    z, t = masked_logits(6, 300, torch.float32, 1.0, 6)
    t[:] = torch.tensor([0, 1, 2], device="cuda")
    r = flce.token_logprobs(z, t, -100, 1.0, 0, True)
    g, b, c = torch.ones(6, 3, device="cuda"), torch.ones(6, device="cuda"), torch.ones(6, device="cuda")
    {"logprob": g[4], "entropy": b[4:5], "lse": c[4:5]}[which].fill_(float("nan"))
    d = flce.token_logprobs_backward(z, t, r.stats, r.entropy, None, g, None, b, c)
    assert torch.isnan(d[4]).all() and torch.isfinite(d[[0, 1, 2, 3, 5]]).all()
