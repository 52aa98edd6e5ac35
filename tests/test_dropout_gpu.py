"""Dropout on the GPU against the fp64 definition: the mask exactly, values to their roundings."""
import numpy as np
import pytest

from oracle import block_ref as ref
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x9E3779B97F4A7C15, (1 << 40) + 3


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def rand(M, H, dtype, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, H, generator=gen, device="cuda").to(dt(dtype))


def bound(want, x, r, dtype):
    """x / (1 - q) with the factor rounded once, one fused multiply-add, one store."""
    e = 2 * ou.U32 * (1.5 * np.abs(x) * 2 + np.abs(want))
    return ou.half_step(dtype) * (np.abs(want) + e) + e


@pytest.mark.parametrize("M,H", [(1, 1), (3, 7), (2, 8), (5, 9), (4, 64), (33, 100), (65, 1000), (2, 8191), (257, 24)])
@pytest.mark.parametrize("x,r", [("bf16", None), ("fp32", None), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"),
                                 ("fp32", "fp32")])
def test_against_the_definition(M, H, x, r):
    import torch
    from log_prob_amd import flce
    a = rand(M, H, x, M + H)
    b = None if r is None else rand(M, H, r, M + H + 1)
    a64, b64 = ou.np64(a), None if b is None else ou.np64(b)
    for p in (0.0, 0.1, 0.5):
        want = ref.dropout(a64, p, SEED, OFFSET, b64)
        for out in (None, torch.bfloat16, torch.float32):
            y = flce.dropout(a, p, SEED, OFFSET, b, out)
            assert y.dtype == (out or (a if b is None else b).dtype)
            ou.check_within(ou.np64(y), want, bound(want, a64, b64, y.dtype), f"{M}x{H} {x} {r} {p} {out}")


def test_mask_of_many_rows():
    """A row's mask does not depend on what else is in the call, and its gradient uses the same."""
    import torch
    from log_prob_amd import flce
    M, H, p = 40000, 520, 0.25
    one = torch.ones(M, H, device="cuda")
    y = flce.dropout(one, p, SEED, OFFSET)
    assert torch.equal(y[-300:], flce.dropout(one, p, SEED, OFFSET)[-300:])
    assert torch.equal(y[:300], flce.dropout(one[:300], p, SEED, OFFSET))
    kept = y != 0
    assert torch.equal(y[kept], torch.full_like(y[kept], 1 / 0.75)) and abs(float(kept.float().mean()) - 0.75) < 1e-3
    assert torch.equal(flce.dropout_backward(one, p, SEED, OFFSET, torch.bfloat16) != 0, kept)
    rows = [0, 1, 77, 39999]
    bits = np.array([[h for b in range(H // 8) for w in ref.philox(
        (b, m, OFFSET & 0xFFFFFFFF, OFFSET >> 32), (SEED & 0xFFFFFFFF, SEED >> 32)) for h in (w & 0xFFFF, w >> 16)]
        for m in rows])
    assert np.array_equal(kept[rows].cpu().numpy(), bits >= 16384)


def test_edges_of_p_and_what_is_dropped():
    import torch
    from log_prob_amd import flce
    x = rand(5, 72, "fp32", 3)
    x[0, :], x[1, :] = float("nan"), float("inf")
    r = rand(5, 72, "fp32", 4)
    assert torch.equal(flce.dropout(x, 0.0, 1)[2:], x[2:]) and torch.isnan(flce.dropout(x, 0.0, 1)[0]).all()
    assert torch.equal(flce.dropout(x, 1.0, 1), torch.zeros_like(x))
    assert torch.equal(flce.dropout(x, 1.0, 1, residual=r), r)
    keep = torch.from_numpy(ref.dropout_bits(5, 72, 9, 0) >= 32768).cuda()
    y = flce.dropout(x, 0.5, 9, residual=r)
    assert torch.equal(torch.isfinite(y[:2]), ~keep[:2]) and torch.equal(y[~keep], r[~keep])
    empty = flce.dropout(x[:0], 0.5, 9)
    assert empty.shape == (0, 72)


@pytest.mark.parametrize("H,pad,shift", [(64, 8, 0), (64, 3, 0), (100, 4, 2), (201, 7, 1)])
def test_strides_and_in_place(H, pad, shift):
    import torch
    from log_prob_amd import flce
    M = 9
    x, r = rand(M, H, "bf16", 5), rand(M, H, "bf16", 6)
    want = flce.dropout(x, 0.3, 11, 2, r)

    def wide(t):
        buf = torch.full((M * (H + pad) + shift,), 7.0, dtype=t.dtype, device="cuda")
        view = buf[shift:].view(M, H + pad)[:, :H]
        view.copy_(t)
        return buf, view

    for place in ("out", "x", "residual"):
        bufs = {"x": wide(x), "residual": wide(r), "out": wide(torch.zeros_like(x))}
        got = flce.dropout(bufs["x"][1], 0.3, 11, 2, bufs["residual"][1], out=bufs[place][1])
        assert torch.equal(got, want), place
        for buf, _ in bufs.values():
            assert (buf[shift:].view(M, H + pad)[:, H:] == 7.0).all() and (buf[:shift] == 7.0).all()


def test_seed_in_device_memory():
    import torch
    from log_prob_amd import flce
    x = rand(20, 136, "bf16", 7)
    for seed in (0, 5, (1 << 63) - 1, (1 << 63) + 12345):
        at = torch.tensor([seed - (1 << 64) if seed >> 63 else seed], dtype=torch.int64, device="cuda")
        assert torch.equal(flce.dropout(x, 0.5, at, 4), flce.dropout(x, 0.5, seed, 4))
    assert not torch.equal(flce.dropout(x, 0.5, 5, 4), flce.dropout(x, 0.5, 5, 5))


def test_refusals():
    import torch
    from log_prob_amd import flce
    x = rand(4, 32, "bf16", 1)
    for call in (lambda: flce.dropout(x.double(), 0.1, 1), lambda: flce.dropout(x, 0.1, 1, residual=x.half()),
                 lambda: flce.dropout(x, 0.1, 1, out_dtype=torch.float16),
                 lambda: flce.dropout(x, 0.1, torch.zeros(1, device="cuda")),
                 lambda: flce.dropout(x, 0.1, 1, out=torch.empty(4, 32, device="cuda"), out_dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: flce.dropout(x[0], 0.1, 1), lambda: flce.dropout(x.t(), 0.1, 1),
                 lambda: flce.dropout(x, 0.1, 1, residual=x[:3]), lambda: flce.dropout(x, 0.1, -1),
                 lambda: flce.dropout(x, 0.1, 1, 1 << 64), lambda: flce.dropout(x, 0.1, 1, residual=x.cpu()),
                 lambda: flce.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64, device="cuda")),
                 lambda: flce.dropout(x, 0.1, torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(flce.FlceError):
        flce.dropout(x, 1.5, 1)
