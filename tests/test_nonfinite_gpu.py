"""Infinities and NaNs in a head's operands come out as NaNs: in every output of the rows they
reach, and nowhere else."""
import pytest

pytestmark = pytest.mark.gpu

IGNORE = -100


def same(a, b):
    """The same bits, one NaN as good as another."""
    import torch
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(3.0), b.nan_to_num(3.0))


def check_rows(clean, got, bad, targets):
    """(logprob, lse, entropy or None): NaN in the rows of `bad` (0 where the target is ignored),
    the clean results' bits in the others."""
    import torch
    ignored = targets == IGNORE
    for name, a, b in zip(("logprob", "lse", "entropy"), clean, got):
        if a is None:
            assert b is None
            continue
        want = a.clone()
        want[bad] = float("nan")
        if name != "lse":
            want[ignored] = 0.0
        assert same(b, want), f"{name}: {b[bad][:8].tolist()}"


def fp4_case(M, H, V):
    import torch
    from log_prob_amd import flce
    gen = torch.Generator(device="cuda").manual_seed(7 * M + V)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    X = n(M, H).bfloat16()
    W = flce.mx_quantize((n(V, H) / H ** 0.5).bfloat16(), "mxfp4")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[torch.rand(M, generator=gen, device="cuda") < 0.2] = IGNORE
    t[M // 2] = V - 1
    return X, W, t


# every kernel and merge: tokens quantised by the product itself or beforehand, tiles of up to
# 128 tokens with their partials side by side by token or by tile, and the 256 x 256 tiles
FP4 = [(1, 264, 700), (8, 264, 5000), (40, 264, 700), (140, 264, 700), (1500, 72, 2000),
       (500, 264, 32100), (1100, 264, 40001)]


@pytest.mark.parametrize("ent", [True, False])
@pytest.mark.parametrize("M,H,V", FP4)
def test_fp4_tokens(M, H, V, ent):
    import torch
    from log_prob_amd import flce
    X, W, t = fp4_case(M, H, V)
    clean = flce.mxfp4_forward(X, W, t, IGNORE, compute_entropy=ent)
    assert not any(torch.isnan(v).any() for v in clean if v is not None)
    rows = torch.arange(M, device="cuda")
    bad = (rows == M // 2) | (rows % 97 == 5) | ((t == IGNORE) & (rows % 3 == 0))
    for value in (float("nan"), float("inf"), -float("inf")):
        X2 = X.clone()
        X2[bad, H // 3] = value
        check_rows(clean, flce.mxfp4_forward(X2, W, t, IGNORE, compute_entropy=ent), bad, t)
        z, z2 = flce.mxfp4_logits(X, W), flce.mxfp4_logits(X2, W)
        z[bad] = float("nan")
        assert same(z2, z)


@pytest.mark.parametrize("scale", [1.0, -0.5])
@pytest.mark.parametrize("M,H,V", FP4)
def test_fp4_weights(M, H, V, scale):
    """One block of W without a number (scale byte 255): its word's logits, and so every sum
    over the vocabulary.  A token of zeros is no exception."""
    import torch
    from log_prob_amd import flce
    X, W, t = fp4_case(M, H, V)
    X[M // 2] = 0.0
    clean = flce.mxfp4_forward(X, W, t, IGNORE, scale)
    z = flce.mxfp4_logits(X, W, scale)
    for word in (0, V // 2, V - 1):
        scales = W.scales.clone()
        scales[word, 3 % (H // 32)] = 255
        W2 = W._replace(scales=scales)
        check_rows(clean, flce.mxfp4_forward(X, W2, t, IGNORE, scale),
                   torch.ones(M, dtype=torch.bool, device="cuda"), t)
        want = z.clone()
        want[:, word] = float("nan")
        assert same(flce.mxfp4_logits(X, W2, scale), want)
