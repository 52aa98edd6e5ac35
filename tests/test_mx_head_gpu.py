"""The head with 4-bit weights on the GPU against the fp64 definition.

Products of e2m1 codes are exact, so a logit's only errors are those of its fp32 sum: H
additions, each off by at most a step (2^-23, should the matrix unit not round to nearest) of
a partial sum no larger than the sum of magnitudes, and the rounding of the output."""
import numpy as np
import pytest

from oracle import ops_ref as ops
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

IGNORE = -100


def make(M, H, V, seed, x_scale=1.0):
    import torch
    from log_prob_amd import flce
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    X = (x_scale * n(M, H)).bfloat16()
    W = flce.mx_quantize((n(V, H) / H ** 0.5).bfloat16(), "mxfp4")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t = torch.where(torch.rand(M, generator=gen, device="cuda") < 0.1, IGNORE, t)
    return X, W, t


def reference(X, W, scale):
    """fp64 logits and the elementwise bound of an fp32 sum's error."""
    import torch
    from log_prob_amd import flce
    Wv = ou.np64(flce.mx_dequantize(W, torch.float32))
    Xv = ops.rounded(ou.np64(X), "mxfp4")
    s = float(np.float32(scale))
    z = s * (Xv @ Wv.T)
    e = abs(s) * (X.shape[1] + 2) * 2 * ou.U32 * (np.abs(Xv) @ np.abs(Wv).T)
    return Wv, z, e


def check_logits(X, W, scale, label, out=None):
    import torch
    from log_prob_amd import flce
    _, z, e = reference(X, W, scale)
    for dtype in (torch.float32, torch.bfloat16):
        got = flce.mxfp4_logits(X, W, scale, out_dtype=dtype)
        assert got.dtype == dtype
        half = ou.half_step(dtype)
        ou.check_within(ou.np64(got), z, half * (np.abs(z) + e) + e, f"{label} {dtype}")


def forward_bounds(z, e, V):
    """Bounds of (logprob, lse, entropy) from those of the logits: the shifted exponentials'
    arguments round relative to the largest logit, their sums add V / 256 tiles of 256."""
    ez = e.max(axis=1)
    big = np.abs(z).max(axis=1)
    spread = z.max(axis=1) - z.min(axis=1)
    e_lse = ez + ou.U32 * (16 * big + V / 256 + 128)
    e_ent = ez * (2 + spread) + ou.U32 * (16 * (big + 1) * (1 + spread) + (spread + 8) * (V / 256 + 128))
    return ez + e_lse, e_lse, e_ent


def check_forward(X, W, t, scale, label, ent=True, **kw):
    from log_prob_amd import flce
    Wv, z, e = reference(X, W, scale)
    want = ops.fp4_forward(ou.np64(X), Wv, t.cpu().numpy(), IGNORE, scale)
    e_lp, e_lse, e_ent = forward_bounds(z, e, z.shape[1])
    lp, lse, en = flce.mxfp4_forward(X, W, t, IGNORE, scale, ent, **kw)
    ou.check_within(ou.np64(lp), want["logprob"], e_lp, f"{label} logprob")
    ou.check_within(ou.np64(lse), want["lse"], e_lse, f"{label} lse")
    assert (lp <= 0).all() and (lp[t == IGNORE] == 0).all()
    if ent:
        ou.check_within(ou.np64(en), want["entropy"], e_ent, f"{label} entropy")
        assert (en >= 0).all()
    else:
        assert en is None
    return lp, lse, en


# one token to several row tiles, one word to several vocabulary tiles, hidden sizes that end
# inside a block, a step, a pair of steps
SHAPES = [(1, 8, 1), (1, 32, 40), (2, 24, 33), (1, 256, 1000), (3, 248, 255), (5, 264, 256),
          (31, 40, 257), (32, 512, 300), (33, 520, 513), (64, 1000, 1003), (65, 768, 700),
          (127, 136, 2000), (128, 1032, 511), (129, 2056, 260), (200, 64, 5003), (256, 288, 1024),
          (257, 544, 769), (300, 4096, 530), (513, 320, 1500), (1, 8192, 777), (700, 128, 50257),
          # few tokens, quantised by the product itself or beforehand, over vocabularies that
          # give a workgroup 32, 64 and 128 rows
          (8, 2048, 1400), (8, 2080, 500), (7, 4096, 300), (2, 8200, 100), (1, 16392, 70),
          (5, 520, 25000), (8, 2568, 24600), (30, 264, 25001), (50, 136, 24999), (1, 264, 50257),
          (8, 520, 50000), (8, 3080, 49200), (20, 136, 50257), (64, 136, 50000), (100, 72, 50257),
          # more tokens in tiles of 64, 96 and 128, past 1024 tokens, and over vocabularies that
          # take the 256 x 256 tiles
          (130, 2056, 1003), (600, 136, 700), (200, 264, 30001), (257, 520, 30000), (400, 264, 33000),
          (1500, 72, 2000), (512, 72, 32501), (500, 776, 32003), (1000, 520, 16101), (1280, 40, 13001)]


@pytest.mark.parametrize("M,H,V", SHAPES)
def test_shapes(M, H, V):
    X, W, t = make(M, H, V, 100 * M + H)
    check_logits(X, W, 1.0, f"{M}x{H}x{V}")
    check_forward(X, W, t, 1.0, f"{M}x{H}x{V}")


@pytest.mark.parametrize("scale", [1 / 0.7, -0.5, 0.0, 37.0])
@pytest.mark.parametrize("M,V", [(4, 1300), (70, 1300), (150, 1300), (300, 40000), (500, 32100)])
def test_scales(M, V, scale):
    X, W, t = make(M, 200, V, M)
    check_logits(X, W, scale, f"scale {scale}")
    check_forward(X, W, t, scale, f"scale {scale}")
    check_forward(X, W, t, scale, f"scale {scale}", ent=False)


@pytest.mark.parametrize("M", [7, 140, 300])
def test_rows_of_every_magnitude(M):
    """Tokens from 2^-100 to 2^100 and a zero row: the block scales carry the range."""
    import torch
    X, W, t = make(M, 320, 900, 5)
    m = torch.pow(2.0, torch.linspace(-100, 100, M, device="cuda"))
    m[M // 2] = 0.0
    X = (X.float() * m[:, None]).bfloat16()
    _, z, e = reference(X, W, 1.0)
    from log_prob_amd import flce
    ou.check_within(ou.np64(flce.mxfp4_logits(X, W, out_dtype=torch.float32)), z,
                    ou.U32 * (np.abs(z) + e) + e, "magnitudes")


@pytest.mark.parametrize("M,V", [(1, 700), (40, 700), (140, 700), (300, 40000), (500, 32100)])
def test_nonfinite_tokens_stay_in_their_rows(M, V):
    import torch
    from log_prob_amd import flce
    X, W, t = make(M, 264, V, 8)
    X2 = X.clone()
    X2[M // 2, 100] = float("inf")
    for f in (lambda x: flce.mxfp4_logits(x, W), lambda x: flce.mxfp4_forward(x, W, t.clamp(min=0))[1]):
        a, b = f(X), f(X2)
        keep = torch.arange(M, device="cuda") != M // 2
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[M // 2]).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,V,pad,shift", [(3, 1000, 24, 0), (3, 1001, 0, 0), (300, 1001, 7, 0),
                                           (300, 1000, 8, 8), (260, 515, 0, 1), (300, 999, 1, 3),
                                           (129, 1000, 4, 0), (500, 32000, 8, 8), (500, 32001, 7, 0),
                                           (512, 32003, 1, 3), (300, 40001, 2, 1)])
def test_output_strides(M, V, pad, shift, dtype):
    """Rows inside wider rows, at any natural alignment; what lies between is left alone."""
    import torch
    from log_prob_amd import flce
    X, W, _ = make(M, 136, V, 9)
    ref = flce.mxfp4_logits(X, W, 0.5, out_dtype=getattr(torch, dtype))
    buf = torch.full((M * (V + pad) + shift + 64,), 7.0, dtype=ref.dtype, device="cuda")
    out = buf[shift:shift + M * (V + pad)].view(M, V + pad)[:, :V]
    flce.mxfp4_logits(X, W, 0.5, out=out)
    assert torch.equal(out, ref)
    assert (buf[:shift] == 7.0).all() and (buf[shift + M * (V + pad):] == 7.0).all()
    assert (buf[shift:shift + M * (V + pad)].view(M, V + pad)[:, V:] == 7.0).all()


@pytest.mark.parametrize("H,V,M", [(264, 1700, 1000), (512, 300, 520), (72, 20000, 2500), (264, 16000, 1000),
                                   (72, 13000, 1280)])
def test_waves_give_the_same_bits(H, V, M):
    """Any workspace from one 256-row wave up; stale and guard bytes do not matter."""
    import torch
    from log_prob_amd import flce
    X, W, t = make(M, H, V, 11)
    ref = check_forward(X, W, t, 1.0, "one wave")
    full = flce.mxfp4_workspace_query(M, H, V)[1]

    def takes(n):
        try:
            flce.mxfp4_forward(X, W, t, IGNORE, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        except flce.FlceError as err:
            assert err.status == 3
            return False
        return True

    # the smallest workspace that is accepted, a wave of at most 256 rows
    none, least = 0, full
    while least - none > 1:
        mid = (none + least) // 2
        none, least = (none, mid) if takes(mid) else (mid, least)
    assert least <= full // 2 + 256
    for n in (full, full - 1, (full + least) // 2, least):
        ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        got = flce.mxfp4_forward(X, W, t, IGNORE, workspace=ws[:n])
        for a, b in zip(got, ref):
            assert torch.equal(a, b), n
        assert (ws[n:] == 0xFF).all()
    with pytest.raises(flce.FlceError) as err:
        flce.mxfp4_forward(X, W, t, IGNORE, workspace=ws[:least - 1])
    assert err.value.status == 3


def test_targets_outside_the_vocabulary():
    import torch
    from log_prob_amd import flce
    X, W, t = make(6, 136, 500, 13)
    t = torch.tensor([499, 500, -1, IGNORE, 1 << 40, 0], device="cuda")
    lp, lse, ent = check_forward(X, W, t, 1.0, "targets")
    assert (lp[1:5] == 0).all() and (ent[1:5] == 0).all() and torch.isfinite(lse).all()


def test_no_tokens_and_one_word():
    import torch
    from log_prob_amd import flce
    X, W, t = make(5, 64, 1, 14)
    check_forward(X, W, torch.zeros_like(t), 1.0, "one word")   # log-prob and entropy of 0
    X0 = X[:0].contiguous()
    assert flce.mxfp4_logits(X0, W).shape == (0, 1)
    assert flce.mxfp4_forward(X0, W, t[:0])[0].shape == (0,)


def test_a_row_does_not_depend_on_its_batch():
    """The same token alone, in a small batch and in a large one: the same logits."""
    import torch
    from log_prob_amd import flce
    X, W, t = make(600, 1032, 1300, 15)
    all_ = flce.mxfp4_logits(X, W, out_dtype=torch.float32)
    _, z, e = reference(X, W, 1.0)
    for n in (1, 40, 100, 130, 300):
        part = flce.mxfp4_logits(X[:n].contiguous(), W, out_dtype=torch.float32)
        ou.check_within(ou.np64(part), z[:n], ou.U32 * np.abs(z[:n]) + e[:n], f"{n} tokens")
        assert float((part - all_[:n]).abs().max()) <= 2 * float(e.max())


def test_refusals():
    import torch
    from log_prob_amd import flce
    X, W, t = make(4, 64, 100, 16)
    with pytest.raises(TypeError):
        flce.mxfp4_logits(X.float(), W)
    with pytest.raises(ValueError):
        flce.mxfp4_logits(X[:, :32], W)
    with pytest.raises(ValueError):
        flce.mxfp4_logits(X[:, :32].contiguous(), W)
    with pytest.raises(ValueError):
        flce.mxfp4_logits(X, flce.mx_quantize(X, "mxfp8"))
    with pytest.raises(ValueError):
        flce.mxfp4_logits(X, W._replace(scales=W.scales[:, :2]))
    with pytest.raises(TypeError):
        flce.mxfp4_logits(X, W, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        flce.mxfp4_forward(X, W, t.int())
    with pytest.raises(ValueError):
        flce.mxfp4_forward(X, W, t[:3])
    with pytest.raises(flce.FlceError) as err:
        flce.mxfp4_logits(X, W, scale=float("nan"))
    assert err.value.status == 1
    x4 = torch.zeros(4, 60, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(flce.FlceError) as err:
        flce.mxfp4_logits(x4, flce.mx_quantize(x4, "mxfp4"))
    assert err.value.status == 2
