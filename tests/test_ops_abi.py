"""Refusals of the layer norm and microscaled calls: all of them on the host, before any HIP
call, so no device is needed (pointers are never followed)."""
import pytest

from log_prob_amd import flce

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3
P = 1 << 20   # an address that is only looked at


def status(name, *args):
    return getattr(flce.load(), name)(*args)


def norm_forward(**kw):
    a = dict(x=P, xd=0, ldx=64, w=P, b=P, pd=0, M=4, H=64, eps=1e-5, y=P, yd=0, ldy=64, mean=P,
             rstd=P, fmt=-1, codes=None, scales=None)
    a.update(kw)
    return status("flce_layer_norm_forward", *a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(H=0)), (UNSUPPORTED, dict(M=(1 << 30) + 1)),
    (UNSUPPORTED, dict(H=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21)),
    (INVALID, dict(xd=2)), (INVALID, dict(yd=-1)), (INVALID, dict(pd=7)),
    (UNSUPPORTED, dict(xd=0, yd=1)), (INVALID, dict(eps=-1e-5)), (INVALID, dict(eps=float("nan"))),
    (INVALID, dict(eps=float("inf"))), (INVALID, dict(fmt=0, codes=P, scales=P)),
    (INVALID, dict(fmt=5, codes=P, scales=P)), (INVALID, dict(fmt=1)),
    (INVALID, dict(fmt=2, codes=P)), (UNSUPPORTED, dict(fmt=2, codes=P + 8, scales=P)),
    (INVALID, dict(x=None)), (INVALID, dict(y=None)), (INVALID, dict(mean=None)),
    (INVALID, dict(rstd=None)), (INVALID, dict(ldx=63)), (INVALID, dict(ldy=0)),
    (UNSUPPORTED, dict(ldx=(1 << 40) + 1)), (UNSUPPORTED, dict(x=P + 1)),
    (UNSUPPORTED, dict(xd=1, x=P + 2)), (UNSUPPORTED, dict(w=P + 1)),
    (UNSUPPORTED, dict(pd=1, b=P + 2)), (UNSUPPORTED, dict(mean=P + 2)),
])
def test_layer_norm_forward(want, kw):
    assert norm_forward(**kw) == want
    assert flce.load().flce_last_error_message()


def norm_backward(**kw):
    a = dict(dy=P, dyd=0, lddy=64, x=P, xd=0, ldx=64, fmt=-1, codes=None, scales=None, w=P, pd=0,
             mean=P, rstd=P, M=4, H=64, dx=P, dxd=0, lddx=64, dw=P, db=P, ws=P, wsb=1 << 20)
    a.update(kw)
    return status("flce_layer_norm_backward", *a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(H=-8)), (INVALID, dict(dyd=3)), (INVALID, dict(xd=3)),
    (INVALID, dict(dxd=3)), (INVALID, dict(pd=3)),
    (INVALID, dict(fmt=1, codes=P, scales=P)),              # x and a checkpoint
    (INVALID, dict(x=None)),                                # neither
    (INVALID, dict(x=None, fmt=0, codes=P, scales=P)),      # no 4-bit checkpoints
    (INVALID, dict(x=None, fmt=1)), (UNSUPPORTED, dict(x=None, fmt=1, codes=P, scales=P + 4)),
    (UNSUPPORTED, dict(xd=1)), (UNSUPPORTED, dict(dyd=1)), (INVALID, dict(dy=None)),
    (INVALID, dict(mean=None)), (INVALID, dict(dx=None)), (INVALID, dict(ws=None)),
    (INVALID, dict(lddy=8)), (INVALID, dict(lddx=8)), (INVALID, dict(ldx=8)),
    (UNSUPPORTED, dict(ws=P + 64)), (TOO_SMALL, dict(wsb=2 * 4 * 64 - 1)),
    (UNSUPPORTED, dict(dw=P + 1)), (UNSUPPORTED, dict(rstd=P + 1)),
])
def test_layer_norm_backward(want, kw):
    assert norm_backward(**kw) == want


def test_layer_norm_workspace():
    assert flce.layer_norm_backward_workspace(0, 64) == 0
    assert flce.layer_norm_backward_workspace(1, 64) == 2 * 4 * 64
    # bounded, whatever the number of rows
    assert (flce.layer_norm_backward_workspace(1 << 30, 4096)
            == flce.layer_norm_backward_workspace(1 << 20, 4096) <= 1024 * 2 * 4 * 4096)
    with pytest.raises(flce.FlceError):
        flce.layer_norm_backward_workspace(1, 0)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)), (UNSUPPORTED, dict(cols=(1 << 20) + 1)),
    (INVALID, dict(xd=2)), (INVALID, dict(fmt=-1)), (INVALID, dict(fmt=3)), (INVALID, dict(x=None)),
    (INVALID, dict(ldx=31)), (UNSUPPORTED, dict(x=P + 1)), (INVALID, dict(codes=None)),
    (INVALID, dict(scales=None)), (UNSUPPORTED, dict(codes=P + 8)), (UNSUPPORTED, dict(scales=P + 1)),
])
def test_quantize(want, kw):
    a = dict(x=P, xd=0, ldx=32, rows=2, cols=32, fmt=0, codes=P, scales=P)
    a.update(kw)
    assert status("flce_mx_quantize", *a.values(), None) == want
    d = dict(codes=a["codes"], scales=a["scales"], fmt=a["fmt"], rows=a["rows"], cols=a["cols"],
             out=a["x"], od=a["xd"], ldo=a["ldx"])
    assert status("flce_mx_dequantize", *d.values(), None) == want


def test_sizes():
    assert flce.mx_sizes(1, "mxfp4") == (16, 16)
    assert flce.mx_sizes(32, "mxfp8") == (32, 16)
    assert flce.mx_sizes(513, "mxint8") == (544, 32)
    assert flce.mx_sizes(512, "mxfp4") == (256, 16)
    with pytest.raises(ValueError):
        flce.mx_sizes(32, "fp4")
    for cols, fmt in ((0, "mxfp8"), ((1 << 20) + 1, "mxfp4")):
        with pytest.raises(flce.FlceError):
            flce.mx_sizes(cols, fmt)
    # the binding's own arithmetic is the library's
    for cols in (1, 31, 32, 33, 511, 512, 513, 4096, 10007):
        for fmt, f in flce.MX_FORMATS.items():
            assert flce._mx_row_bytes(cols, f) == flce.mx_sizes(cols, fmt)


def test_empty_calls_touch_nothing():
    assert norm_forward(M=0, x=None, y=None, mean=None, rstd=None) == 0
    assert norm_backward(M=0, dy=None, x=None, dx=None, mean=None, rstd=None, ws=None, wsb=0, dw=None,
                         db=None) == 0
    assert status("flce_mx_quantize", None, 0, 32, 0, 32, 0, None, None, None) == 0
    assert status("flce_mx_dequantize", None, None, 0, 0, 32, None, 0, 32, None) == 0


def test_compiled_binding_declines_host_tensors():
    import torch
    nat = flce._fast()
    x, v = torch.zeros(2, 32), torch.zeros(2)
    u = torch.zeros(2, 16, dtype=torch.uint8)
    assert nat.layer_norm_forward(x, None, None, 1e-5, None, -1) is None
    assert nat.layer_norm_backward(x, x, None, None, -1, v, v, None, None, True, None) is None
    assert nat.mx_quantize(x, 0) is None and nat.mx_dequantize(u, u, 0, 32, None) is None
    assert nat.mxfp4_logits(x.bfloat16(), u, u, 1.0, None) is None
    assert nat.mxfp4_forward(x.bfloat16(), u, u, v.long(), -100, 1.0, True) is None
    assert nat.mx_quantize() is None and nat.mx_quantize(1, 2, 3) is None


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    x = torch.zeros(2, 32)
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x)
    with pytest.raises(ValueError):
        flce.mx_quantize(x, "mxfp4")
    with pytest.raises(ValueError):
        flce.mx_quantize(x, "int4")


def logits(**kw):
    a = dict(X=P, wc=P, ws=P, M=20, H=64, V=100, scale=1.0, out=P, od=0, ldo=100, work=P, wb=1 << 20)
    a.update(kw)
    return status("flce_mx_logits", *a.values(), None)


def mx_forward(**kw):
    a = dict(X=P, wc=P, ws=P, t=P, M=20, H=64, V=100, ignore=-100, scale=1.0, ent=1, lp=P, lse=P, en=P,
             work=P, wb=1 << 24)
    a.update(kw)
    return status("flce_mx_forward", *a.values(), None)


HEAD = [(INVALID, dict(M=-1)), (INVALID, dict(H=0)), (INVALID, dict(V=0)), (UNSUPPORTED, dict(H=60)),
        (UNSUPPORTED, dict(M=(1 << 30) + 1)), (INVALID, dict(scale=float("inf"))),
        (INVALID, dict(X=None)), (INVALID, dict(wc=None)), (INVALID, dict(ws=None)),
        (UNSUPPORTED, dict(X=P + 8)), (UNSUPPORTED, dict(wc=P + 8)), (UNSUPPORTED, dict(ws=P + 4)),
        (INVALID, dict(work=None)), (UNSUPPORTED, dict(work=P + 16)), (TOO_SMALL, dict(wb=100))]


@pytest.mark.parametrize("want,kw", HEAD + [
    (INVALID, dict(od=2)), (INVALID, dict(out=None)), (INVALID, dict(ldo=99)),
    (UNSUPPORTED, dict(ldo=(1 << 40) + 1)), (UNSUPPORTED, dict(out=P + 1)),
    (UNSUPPORTED, dict(od=1, out=P + 2))])
def test_mx_logits(want, kw):
    assert logits(**kw) == want


@pytest.mark.parametrize("want,kw", HEAD + [
    (INVALID, dict(ent=2)), (INVALID, dict(t=None)), (INVALID, dict(lp=None)), (INVALID, dict(lse=None)),
    (INVALID, dict(en=None)), (UNSUPPORTED, dict(t=P + 4)), (UNSUPPORTED, dict(lse=P + 2))])
def test_mx_forward(want, kw):
    assert mx_forward(**kw) == want


def test_mx_workspace():
    # a decoding step's tokens need no copy of their own, only the partials of the forward: 4
    # workgroups of 32 vocabulary rows for 4 tokens, 3 arrays, and counters
    lo, fw = flce.mxfp4_workspace_query(4, 64, 100)
    assert (lo, fw) == (0, 3 * 256 + 256)
    assert mx_forward(M=4, wb=fw - 1) == TOO_SMALL
    # more tokens do: 32 bytes of codes and 16 of scales a row, each part rounded up to 256
    lo, fw = flce.mxfp4_workspace_query(20, 64, 100)
    assert lo == 768 + 512 and fw == lo + 3 * 512 + 256
    assert mx_forward(M=20, wb=fw - 1) == TOO_SMALL and logits(M=20, wb=lo - 1) == TOO_SMALL
    # past 1024 tokens in small tiles: partials of 256-row multiples
    lo, fw = flce.mxfp4_workspace_query(1500, 64, 2000, False)
    assert lo == 1500 * 32 + 128 + 1500 * 16 + 64
    assert fw == lo + 2 * 4 * 16 * 1536 + 256
    # 256 x 256 tiles: whole scale tiles of X
    lo, fw = flce.mxfp4_workspace_query(500, 64, 32000, False)
    assert lo == 500 * 32 + 128 + 512 * 16
    assert fw == lo + 2 * 4 * 125 * 512 + 256
    # and past 2.5e11 products a copy of W's scales
    lo, _ = flce.mxfp4_workspace_query(4096, 4096, 32768)
    assert lo == 32768 * 128 + 4096 * (2048 + 128)
    assert flce.mxfp4_workspace_query(0, 64, 100) == (0, 0)
    assert mx_forward(M=0, X=None, t=None, lp=None, lse=None, en=None, work=None, wb=0) == 0
    assert logits(M=0, X=None, out=None, work=None, wb=0) == 0
