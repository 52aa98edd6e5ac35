"""4-bit calls large enough to re-order W's scales for the 256 x 256 tiles (2048 tokens and
2.5e11 products on), against fp64 on the GPU.

The operands' values are those of mx_dequantize, which is tested byte for byte elsewhere; the
bounds are those of the head's other tests: H + 2 additions of exact products, each off by at
most a step (2^-23) of a partial sum no larger than the sum of magnitudes, one rounding of the
output; the shifted exponentials' arguments round relative to the largest logit and V / 256
tiles of 256 are added."""
import pytest

from tests import ops_util as ou

pytestmark = pytest.mark.gpu

IGNORE = -100
# tokens in whole tiles and not, hidden sizes with an odd and an even number of 16-byte pieces of
# scales and a last step that is part of a pair, vocabularies that end inside a tile
SHAPES = [(2048, 8200, 15003), (2309, 4104, 26500), (4100, 1056, 57857), (2560, 16384, 6001)]


@pytest.fixture(autouse=True)
def room():
    import gc
    import torch
    yield
    gc.collect()
    torch.cuda.empty_cache()


def make(M, H, V):
    """X, W, targets; every scale byte of W's first columns differs between rows and blocks."""
    import torch
    from log_prob_amd import flce
    gen = torch.Generator(device="cuda").manual_seed(M + H)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    X = n(M, H).bfloat16()
    blocks = torch.pow(2.0, torch.randint(-4, 5, (V, -(-H // 32)), generator=gen, device="cuda"))
    W = flce.mx_quantize(n(V, H) / H ** 0.5 * blocks.repeat_interleave(32, 1)[:, :H], "mxfp4")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[torch.rand(M, generator=gen, device="cuda") < 0.1] = IGNORE
    t[0], t[M - 1] = V - 1, 0
    sb = flce.mx_sizes(H, "mxfp4")[1]
    lo, full = flce.mxfp4_workspace_query(M, H, V)
    turned = -(-V // 256) * 256 * sb
    assert lo >= turned + M * sb, "the call does not re-order W's scales"
    return X, W, t, turned, full


def reference(X, W):
    """fp64 logits at scale 1 and the bound of the fp32 sums."""
    import torch
    from log_prob_amd import flce
    Xv = flce.mx_dequantize(flce.mx_quantize(X, "mxfp4"), torch.float32).double()
    Wv = flce.mx_dequantize(W, torch.float32).double().t().contiguous()
    e = (X.shape[1] + 2) * 2 * ou.U32 * (Xv.abs() @ Wv.abs())
    return Xv @ Wv, e


def within(got, want, bound, label):
    assert got.shape == want.shape
    over = (got.double() - want).abs() - bound
    assert not (over > 0).any() and got.isfinite().all(), f"{label}: {float(over.max())} past the bound"


@pytest.mark.parametrize("M,H,V", SHAPES)
def test_logits(M, H, V):
    import torch
    from log_prob_amd import flce
    X, W, _, _, _ = make(M, H, V)
    z, e = reference(X, W)
    for scale, dtype, pad in ((1.0, torch.float32, 0), (-0.75, torch.bfloat16, 0), (0.5, torch.bfloat16, 5)):
        buf = torch.full((M, V + pad), 7.0, dtype=dtype, device="cuda")
        flce.mxfp4_logits(X, W, scale, out=buf[:, :V])
        b = abs(scale) * e
        within(buf[:, :V], scale * z, ou.half_step(dtype) * ((scale * z).abs() + b) + b, f"{scale} {dtype}")
        assert (buf[:, V:] == 7.0).all()


@pytest.mark.parametrize("scale", [1.0, -0.5])
@pytest.mark.parametrize("M,H,V", SHAPES)
def test_forward_whole_and_in_waves(M, H, V, scale):
    """All rows at once, and in waves of which only the first re-orders: the same bits, from any
    stale workspace, with nothing written past its end."""
    import torch
    from log_prob_amd import flce
    X, W, t, turned, full = make(M, H, V)
    z, e = reference(X, W)
    z, e = z * scale, e * abs(scale)
    got = flce.mxfp4_forward(X, W, t, IGNORE, scale)
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    ent = lse - (p * z).sum(1)
    valid = t != IGNORE
    at = torch.arange(M, device="cuda")
    zt = z[at, t.clamp(min=0)]
    zero = torch.zeros_like(lse)
    big, ez, spread = z.abs().amax(1), e.amax(1), z.amax(1) - z.amin(1)
    e_lse = ez + ou.U32 * (16 * big + V / 256 + 128)
    e_ent = ez * (2 + spread) + ou.U32 * (16 * (big + 1) * (1 + spread) + (spread + 8) * (V / 256 + 128))
    within(got[0], torch.where(valid, zt - lse, zero), ez + e_lse, "logprob")
    within(got[1], lse, e_lse, "lse")
    within(got[2], torch.where(valid, ent, zero), e_ent, "entropy")
    plain = flce.mxfp4_forward(X, W, t, IGNORE, scale, False)
    assert torch.equal(plain[0], got[0]) and torch.equal(plain[1], got[1]) and plain[2] is None
    one = flce.mxfp4_workspace_query(256, H, V)[1]   # more than a wave's share, W's copy aside
    for n in (full, (full + turned) // 2, turned + 2 * one):
        n = min(n, full) // 256 * 256
        ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        again = flce.mxfp4_forward(X, W, t, IGNORE, scale, workspace=ws[:n])
        assert all(torch.equal(a, b) for a, b in zip(again, got)), n
        assert (ws[n:] == 0xFF).all()
    with pytest.raises(flce.FlceError) as err:
        flce.mxfp4_forward(X, W, t, IGNORE, scale, workspace=ws[:turned])
    assert err.value.status == 3


def test_graph_replays():
    """Logits and a forward in waves captured with one workspace between them; W's scales change
    between the replays, in place."""
    import torch
    from log_prob_amd import flce
    M, H, V = 2309, 4104, 26500
    X, W, t, turned, full = make(M, H, V)
    ws = torch.empty((full + turned) // 2 // 256 * 256, dtype=torch.uint8, device="cuda")
    wl = torch.empty(flce.mxfp4_workspace_query(M, H, V)[0], dtype=torch.uint8, device="cuda")
    out = tuple(torch.empty(M, device="cuda") for _ in range(3))
    z = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")

    def step():
        flce.mxfp4_logits(X, W, workspace=wl, out=z)
        flce.mxfp4_forward(X, W, t, IGNORE, workspace=ws, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        W.scales.copy_(W.scales.roll(1, 0))
        step()
        want = [v.clone() for v in (z, *out)]
        for v in (z, *out):
            v.zero_()
        ws.fill_(0xFF)
        wl.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((z, *out), want)), f"replay {i}"
