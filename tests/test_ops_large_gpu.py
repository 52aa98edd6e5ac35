"""Layer norm, the quantiser and the 4-bit head on matrices whose offsets pass 32 bits: the
last rows against the same rows in a call of their own."""
import pytest

from tests import ops_util as ou

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(autouse=True)
def room():
    """These tests hold up to 20 GB: give back what is cached on both sides."""
    import gc
    import torch
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_layer_norm_and_checkpoint():
    """300000 x 8192 bf16: 2.5e9 elements, 4.9e9 bytes."""
    import torch
    from log_prob_amd import flce
    M, H, n = 300000, 8192, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, H, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(H, generator=gen, device="cuda")
    y, mean, rstd, kept = flce.layer_norm_forward(x, w, None, EPS, checkpoint="mxint8")
    tail = x[-n:].clone()
    y2, mean2, rstd2, kept2 = flce.layer_norm_forward(tail, w, None, EPS, checkpoint="mxint8")
    for a, b in ((y, y2), (mean, mean2), (rstd, rstd2), (kept.codes, kept2.codes), (kept.scales, kept2.scales)):
        assert torch.equal(a[-n:], b)
    back = flce.mx_dequantize(kept)
    assert torch.equal(back[-n:], flce.mx_dequantize(kept2))
    del back
    want = flce.layer_norm_backward(y2, tail, mean2, rstd2, w)[0]
    dx, dw, db = flce.layer_norm_backward(y, x, mean, rstd, w)
    assert torch.equal(dx[-n:], want)
    del dx
    assert torch.isfinite(dw).all() and torch.isfinite(db).all()
    want = flce.layer_norm_backward(y2, kept2, mean2, rstd2, w)[0]
    assert torch.equal(flce.layer_norm_backward(y, kept, mean, rstd, w)[0][-n:], want)
    q = flce.mx_quantize(x, "mxint8")
    assert torch.equal(q.codes, kept.codes) and torch.equal(q.scales, kept.scales)


def test_logits_rows():
    """16700 x 151936 logits (2.5e9) and few rows far apart."""
    import torch
    from log_prob_amd import flce
    M, H, V, n = 16700, 64, 151936, 1100
    gen = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(M, H, generator=gen, device="cuda").bfloat16()
    W = flce.mx_quantize(torch.randn(V, H, generator=gen, device="cuda"), "mxfp4")
    z = flce.mxfp4_logits(X, W)
    tail = X[-n:].contiguous()
    part = flce.mxfp4_logits(tail, W)
    assert torch.equal(z[-n:], part)
    del z
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    for a, b in zip(flce.mxfp4_forward(X, W, t), flce.mxfp4_forward(tail, W, t[-n:].contiguous())):
        assert torch.equal(a[-n:], b)
    far = torch.empty(100, 1 << 26, dtype=torch.bfloat16, device="cuda")[:, :V]
    few = tail[:100].contiguous()
    flce.mxfp4_logits(few, W, out=far)
    assert torch.equal(far, flce.mxfp4_logits(few, W))


@pytest.mark.parametrize("M", [2, 20, 200])
def test_vocabulary_rows(M):
    """600000 x 16384 codes (4.9e9 bytes), and a slice of the vocabulary as a head of its own."""
    import torch
    from log_prob_amd import flce
    H, V, n = 16384, 600000, 700
    cb, sb = flce.mx_sizes(H, "mxfp4")
    gen = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (V, cb), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(117, 123, (V, sb), generator=gen, device="cuda", dtype=torch.uint8)
    W = flce.MXTensor(codes, scales, "mxfp4", H)
    tail = flce.MXTensor(codes[-n:], scales[-n:], "mxfp4", H)
    X = torch.randn(M, H, generator=gen, device="cuda").bfloat16()
    z = flce.mxfp4_logits(X, W, out_dtype=torch.float32)[:, -n:]
    Xv = flce.mx_dequantize(flce.mx_quantize(X, "mxfp4"), torch.float32)
    Wv = flce.mx_dequantize(tail, torch.float32)
    want = Xv.double() @ Wv.double().T
    # exact products, each in at most H + 2 additions that are off by at most a step
    e = (H + 2) * 2 * ou.U32 * (Xv.double().abs() @ Wv.double().abs().T)
    assert ((z.double() - want).abs() <= e).all()
    assert ((flce.mxfp4_logits(X, tail, out_dtype=torch.float32).double() - want).abs() <= e).all()
    t = torch.arange(V - M, V, device="cuda")
    lp, lse, _ = flce.mxfp4_forward(X, W, t)
    # the target logit from the log-prob: both fp32 values of the size of the lse
    zt = want[torch.arange(M), torch.arange(n - M, n)]
    et = e[torch.arange(M), torch.arange(n - M, n)] + 4 * ou.U32 * (lse.abs() + lp.abs()).double()
    assert ((lp.double() + lse.double() - zt).abs() <= et).all()
