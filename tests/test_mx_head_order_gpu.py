"""Which 4-bit calls give a token the same bits: those that share an order of summation.

Over 384 or more workgroups of 128 vocabulary rows every call of up to 128 tokens sums K in one
wave, in order, whatever tile of tokens it takes and whoever quantises them; the sums over the
vocabulary follow the tiles of 128 rows and one merge.  (The target logit is summed by the merge,
in another order where the tokens are quantised by the product itself: the log-prob may differ in
its last bits there.)"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,V", [(264, 50257), (2056, 49153)])
def test_a_token_alone_and_in_batches(H, V):
    import torch
    from log_prob_amd import flce
    gen = torch.Generator(device="cuda").manual_seed(H)
    X = torch.randn(128, H, generator=gen, device="cuda").bfloat16()
    W = flce.mx_quantize(torch.randn(V, H, generator=gen, device="cuda") / H ** 0.5, "mxfp4")
    t = torch.randint(0, V, (128,), generator=gen, device="cuda")
    z = flce.mxfp4_logits(X, W, out_dtype=torch.float32)
    lp, lse, ent = flce.mxfp4_forward(X, W, t)
    for n in (1, 2, 8, 9, 31, 33, 64, 65, 96, 97, 127):
        part = X[:n].contiguous()
        assert torch.equal(flce.mxfp4_logits(part, W, out_dtype=torch.float32), z[:n]), n
        a, b, c = flce.mxfp4_forward(part, W, t[:n].contiguous())
        assert torch.equal(b, lse[:n]) and torch.equal(c, ent[:n]), n
        assert n <= 8 or torch.equal(a, lp[:n]), n
    one = flce.mxfp4_logits(X[77:78].contiguous(), W, out_dtype=torch.float32)
    assert torch.equal(one, z[77:78])
