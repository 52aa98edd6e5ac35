"""Microscaled formats on the GPU: codes, scales and padding bit for bit against the fp64
definition (a search in the table of representable values)."""
import numpy as np
import pytest

from oracle import ops_ref as ops
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "mxfp8", "mxint8"]


def check(x, fmt):
    """Quantise x on the GPU and compare every byte; then the values in both types."""
    import torch
    from log_prob_amd import flce
    q = flce.mx_quantize(x, fmt)
    codes, exps = ops.quantize(ou.np64(x), fmt)
    want = ou.pack(codes, fmt)
    got = q.codes.cpu().numpy()
    if fmt != "mxint8":   # a negative number may keep its sign when it is rounded to 0
        half = 4 if fmt == "mxfp4" else 8
        clear = lambda c: np.where((c & ((1 << half) - 1)) == 1 << (half - 1), 0, c)
        if fmt == "mxfp4":
            got = clear(got & 15) | (clear(got >> 4) << 4)
        else:
            got = clear(got)
    assert np.array_equal(got, want)
    assert np.array_equal(q.scales.cpu().numpy(), ou.pack_scales(exps))
    v = ops.values(codes, exps, fmt, x.shape[1])
    f = flce.mx_dequantize(q, torch.float32)
    with np.errstate(over="ignore"):   # 4 * 2^126 is past fp32's range: infinity there
        assert np.array_equal(f.cpu().numpy(), v.astype(np.float32), equal_nan=True)
    b = flce.mx_dequantize(q)
    assert torch.equal(b.nan_to_num(1e30), f.to(torch.bfloat16).nan_to_num(1e30))  # one rounding
    return q


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,H", [(1, 1), (2, 7), (3, 8), (1, 31), (4, 32), (3, 33), (5, 100),
                                 (2, 512), (300, 520), (7, 1000), (3, 4099), (2, 8192), (1, 40000)])
def test_shapes(M, H, dtype, fmt):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(100 * M + H)
    x = torch.randn(M, H, generator=gen, device="cuda")
    x = x * 10.0 ** torch.randint(-3, 4, (M, H), generator=gen, device="cuda")
    check(x.to(getattr(torch, dtype)), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_bf16_value_under_the_largest(fmt):
    """Each block opens with the format's largest value, so its scale is 1, and the others run
    through every bf16 value up to it: every rounding and every tie."""
    import torch
    top = ops.grid(fmt)[-1]
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[v.double().abs() <= top]
    v = torch.cat((v, torch.zeros(-len(v) % 31, dtype=v.dtype))).view(-1, 31)
    x = torch.cat((torch.full((v.shape[0], 1), top, dtype=v.dtype), v), 1)
    rows = x.reshape(-1).cuda()
    rows = torch.cat((rows, torch.zeros(-len(rows) % 1024, dtype=rows.dtype, device="cuda")))
    check(rows.view(-1, 1024), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_scale(fmt):
    """Block maxima at and around the border of every scale, down to subnormals."""
    import torch
    top = np.float32(ops.grid(fmt)[-1])
    rows = []
    for e in range(-149, 128):
        with np.errstate(over="ignore", under="ignore"):
            edge = np.float32(np.ldexp(np.float64(top), e))
        for m in (np.nextafter(edge, np.float32(0)), edge, np.nextafter(edge, np.float32(np.inf))):
            if np.isfinite(m):
                rows.append(np.concatenate([[m], -m * np.linspace(0, 1, 31, dtype=np.float32)]))
    check(torch.from_numpy(np.array(rows, np.float32)).cuda(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_zeros_and_nonfinite(fmt):
    import torch
    from log_prob_amd import flce
    x = torch.randn(6, 96, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    x[0] = 0.0
    x[1, 40] = float("nan")
    x[2, 0] = float("inf")
    x[3, 95] = -float("inf")
    x[4] = -0.0
    q = check(x, fmt)
    v = flce.mx_dequantize(q, torch.float32)
    assert not v[0].any() and not v[4].any()
    nan = torch.isnan(v)
    want = torch.zeros_like(nan)
    want[1, 32:64] = want[2, :32] = want[3, 64:] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_every_code_and_scale(fmt):
    import torch
    from log_prob_amd import flce
    n = 16 if fmt == "mxfp4" else 256
    codes = np.tile(np.arange(n).reshape(1, -1, 32) if n > 32 else np.arange(32).reshape(1, 1, 32) % 16,
                    (256, 1, 1))
    if fmt == "mxint8":
        signed = np.where(codes > 127, codes - 256, codes)
    else:
        signed = codes
        if fmt == "mxfp8":   # the two NaN codes are never written
            signed = codes = np.where(codes % 128 == 127, 0, codes)
    exps = np.repeat(np.arange(256)[:, None] - 127, codes.shape[1], axis=1)
    cols = codes.shape[1] * 32
    q = flce.MXTensor(torch.from_numpy(ou.pack(codes, fmt)).cuda(),
                      torch.from_numpy(ou.pack_scales(exps)).cuda(), fmt, cols)
    got = flce.mx_dequantize(q, torch.float32).cpu().numpy()
    with np.errstate(over="ignore"):
        want = ops.values(signed, exps, fmt, cols).astype(np.float32)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,pad,shift", [(72, 8, 0), (72, 5, 0), (72, 8, 1), (1000, 24, 8)])
def test_row_strides_and_guards(H, pad, shift, fmt):
    """Strided input and output; nothing outside codes, scales and the rows is written."""
    import torch
    from log_prob_amd import flce
    M = 5
    x = torch.randn(M, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    ref = check(x, fmt)
    buf = torch.zeros(M * (H + pad) + shift, dtype=torch.bfloat16, device="cuda")
    view = buf[shift:].view(M, H + pad)[:, :H]
    view.copy_(x)
    cb, sb = flce.mx_sizes(H, fmt)
    raw_c = torch.full((M * cb + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    raw_s = torch.full((M * sb + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = flce.MXTensor(raw_c[16:16 + M * cb].view(M, cb), raw_s[16:16 + M * sb].view(M, sb), fmt, H)
    flce.mx_quantize(view, fmt, out=out)
    assert torch.equal(out.codes, ref.codes) and torch.equal(out.scales, ref.scales)
    for raw in (raw_c, raw_s):
        assert (raw[:16] == 0xA5).all() and (raw[-48:] == 0xA5).all()
    buf.fill_(7.0)
    flce.mx_dequantize(out, out=view)
    assert torch.equal(view, flce.mx_dequantize(ref))
    assert (buf[shift:].view(M, H + pad)[:, H:] == 7.0).all() and (buf[:shift] == 7.0).all()


def test_no_rows():
    import torch
    from log_prob_amd import flce
    q = flce.mx_quantize(torch.empty(0, 40, device="cuda"), "mxfp8")
    assert q.codes.shape == (0, 64) and flce.mx_dequantize(q).shape == (0, 40)
