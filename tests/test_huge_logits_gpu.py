"""Logits too large for fp32's shifted exponentials: the outputs are right to the rounding of the
largest logit or NaN, never a made-up number.

The kernels shift by the rounded product of the largest logit and log2 e, so the largest term
itself is 2^r with r up to half a step of that product: 64 at logits of 2^30, past fp32's range
from twice that on."""
import numpy as np
import pytest

from oracle import ops_ref as ops
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


def rows(M, H, seed):
    """Tokens from 1 to 2^60, four to a power of two."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(M, H, generator=gen, device="cuda")
    k = torch.arange(M, device="cuda") % 244 // 4
    return (X * torch.pow(2.0, k.float())[:, None]).bfloat16()


def check(got, z, e, targets, V):
    """z: fp64 logits, e: error of the fp32 sums."""
    lse, lp = ou.np64(got[1]), ou.np64(got[0])
    top = z.max(axis=1)
    want = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    big = np.abs(z).max(axis=1)
    zt = z[np.arange(len(z)), targets.cpu().numpy()]
    bound = e.max(axis=1) + ou.U32 * (16 * big + V / 256 + 128)
    nan = np.isnan(lse)
    assert not nan[big < 2.0 ** 30].any()
    assert (np.isnan(lp) == nan).all() and np.isfinite(lse[~nan]).all()
    assert (np.abs(lse - want)[~nan] <= bound[~nan]).all()
    assert (np.abs(lp - (zt - want))[~nan] <= 2 * bound[~nan]).all()
    if got[2] is not None:
        ent = ou.np64(got[2])
        assert np.isnan(ent[nan]).all() and not np.isnan(ent[big < 2.0 ** 30]).any()
    assert nan.any()   # the rows reach that far


@pytest.mark.parametrize("ent", [True, False])
@pytest.mark.parametrize("M,H,V", [(1, 264, 700), (100, 264, 700), (244, 264, 1300), (1500, 72, 2000),
                                   (500, 264, 32100), (1100, 264, 40001)])
def test_fp4_head(M, H, V, ent):
    import torch
    from log_prob_amd import flce
    X = rows(max(M, 244), H, 1)
    X = X[-M:].contiguous() if M < 244 else X
    gen = torch.Generator(device="cuda").manual_seed(2)
    W = flce.mx_quantize(torch.randn(V, H, generator=gen, device="cuda"), "mxfp4")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    Xv, Wv = ops.rounded(ou.np64(X), "mxfp4"), ou.np64(flce.mx_dequantize(W, torch.float32))
    z, e = Xv @ Wv.T, (H + 2) * 2 * ou.U32 * (np.abs(Xv) @ np.abs(Wv).T)
    got = flce.mxfp4_forward(X, W, t, compute_entropy=ent)
    if M == 1:   # one row of 2^60: whatever it is, no number that is not its own
        assert torch.isnan(got[0]).all() or abs(float(got[1]) - z.max()) <= 32 * ou.U32 * np.abs(z).max()
        return
    check(got, z, e, t, V)


@pytest.mark.parametrize("ent", [True, False])
@pytest.mark.parametrize("M,H,V", [(244, 264, 700), (488, 72, 5001)])
def test_bf16_head(M, H, V, ent):
    import torch
    from log_prob_amd import flce
    X = rows(M, H, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randn(V, H, generator=gen, device="cuda").bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    z = ou.np64(X) @ ou.np64(W).T
    e = (H + 2) * 2 * ou.U32 * (np.abs(ou.np64(X)) @ np.abs(ou.np64(W)).T)
    check(flce.forward(X, W, t, compute_entropy=ent), z, e, t, V)
