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


def bf16_case(M, H, V):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(11 * M + V)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    X, W = n(M, H).bfloat16(), (n(V, H) / H ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[torch.rand(M, generator=gen, device="cuda") < 0.2] = IGNORE
    t[M // 2] = V - 1
    return X, W, t


def shards(X, W, t, ent):
    """The forward in two vocabulary shards, merged."""
    import torch
    from log_prob_amd import flce
    (M, H), V = X.shape, W.shape[0]
    cut = max(1, V // 3)
    parts = [flce.forward_partials_shard(X, W[a:b], t, a, IGNORE, compute_entropy=ent)
             for a, b in ((0, cut), (cut, V))]
    stride = max(p.numel() for p in parts)
    stride = -(-stride // 256) * 256
    gathered = torch.zeros(2 * stride, dtype=torch.uint8, device="cuda")
    for r, p in enumerate(parts):
        gathered[r * stride:r * stride + p.numel()] = p
    return flce.forward_merge_shards(t, [0, cut, V], gathered, stride, IGNORE, ent)


@pytest.mark.parametrize("ent", [True, False])
@pytest.mark.parametrize("M,H,V", [(1, 136, 700), (300, 264, 1300), (600, 72, 5001)])
def test_bf16_head(M, H, V, ent):
    """The bf16 head likewise, through one call, the static scratch and vocabulary shards; what
    hangs on the log-probs sees the NaN."""
    import torch
    from log_prob_amd import flce
    X, W, t = bf16_case(M, H, V)
    rows = torch.arange(M, device="cuda")
    bad = (rows == M // 2) | (rows % 97 == 5) | ((t == IGNORE) & (rows % 3 == 0))
    every = torch.ones_like(bad)
    for f in (lambda x, w: flce.forward(x, w, t, IGNORE, compute_entropy=ent),
              lambda x, w: flce.forward_noalloc(x, w, t, IGNORE, compute_entropy=ent),
              lambda x, w: shards(x, w, t, ent)):
        clean = f(X, W)
        assert not any(torch.isnan(v).any() for v in clean if v is not None)
        for value in (float("nan"), float("inf"), -float("inf")):
            X2 = X.clone()
            X2[bad, H // 3] = value
            got = f(X2, W)
            check_rows(clean, got, bad, t)
        assert torch.isnan(flce.nll_reduce(got[0], t, V, IGNORE)[[0, 2]]).all()
        for word in (0, V - 1):
            W2 = W.clone()
            W2[word, 5] = float("nan")
            check_rows(clean, f(X, W2), every, t)


@pytest.mark.parametrize("on_policy", [False, True])
def test_policy_loss(on_policy):
    """A log-prob, old log-prob or advantage without a number reaches the token's loss, the sum
    and the token's gradient, clipped or not; ignored tokens and the other ones are as before."""
    import torch
    from log_prob_amd import flce
    M, V = 40, 100
    gen = torch.Generator(device="cuda").manual_seed(3)
    lp = -3 * torch.rand(M, generator=gen, device="cuda")
    old = None if on_policy else lp + torch.randn(M, generator=gen, device="cuda")
    adv = torch.randn(M, generator=gen, device="cuda")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[7] = IGNORE
    ignored = t == IGNORE
    clean, clips, sums = flce.policy_loss_reduce(lp, old, adv, t, V, IGNORE)
    grad = flce.policy_loss_grad(lp, old, adv, t, V, sums, IGNORE)
    assert torch.isfinite(clean).all() and torch.isfinite(sums).all()
    for k in range(2 if on_policy else 3):
        args = [lp.clone(), adv.clone(), None if on_policy else old.clone()]
        bad = torch.arange(M, device="cuda") % 9 == 7   # the ignored token among them
        args[k][bad] = float("nan")
        loss, clip, out = flce.policy_loss_reduce(args[0], args[2], args[1], t, V, IGNORE)
        got = flce.policy_loss_grad(args[0], args[2], args[1], t, V, out, IGNORE)
        want, want_grad, want_clip = clean.clone(), grad.clone(), clips.clone()
        want[bad & ~ignored] = want_grad[bad & ~ignored] = float("nan")
        want_clip[bad] = 0
        assert same(loss, want) and same(got, want_grad) and torch.equal(clip, want_clip)
        assert torch.isnan(out[[0, 3]]).all() and out[1] == sums[1] and out[2] == want_clip.sum()
