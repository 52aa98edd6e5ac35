"""The operators around the head as they are used together: a training step through norm,
head and loss; scoring and sampling with a 4-bit head; captured graphs and streams."""
import numpy as np
import pytest

from oracle import flce_ref as ref
from oracle import ops_ref as ops
from synth import inputs
from tests import gpu_util as gu
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

EPS = 1e-5


def norm_case(M, H, seed, dtype="float32"):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = (2 * n(M, H) + 0.5 * n(M, 1)).to(getattr(torch, dtype))
    return x, 1 + 0.1 * n(H), 0.1 * n(H)


@pytest.mark.parametrize("checkpoint", [None, "mxfp8", "mxint8"])
def test_training_step(checkpoint):
    """An fp32 residual stream through norm and head to the mean NLL, all by autograd; dx,
    dweight, dbias against the fp64 chain (the norm's output and the head's gradient in bf16,
    as the head has them) within the head's own tolerance."""
    import torch
    from log_prob_amd import autograd
    M, H, V = 700, 264, 1500
    c = inputs.make_case("together", 501, M, H, V, ignore_frac=0.1, grad_mode="none")
    _, W, t, _, _ = gu.to_dev(c)
    x, w, b = (v.requires_grad_() for v in norm_case(M, H, 3))
    y = autograd.layer_norm(x, w, b, EPS, torch.bfloat16, checkpoint)
    lp = autograd.linear_logprob(y, W, t, c.ignore_index)
    n = int((t != c.ignore_index).sum())
    (-lp.sum() / n).backward()

    x64 = ou.np64(x)
    y64, mean, rstd = ops.layer_norm(x64, ou.np64(w), ou.np64(b), EPS)
    ybits = torch.from_numpy(y64).float().bfloat16()
    glp = np.full(M, -1.0 / n, np.float32)
    dy, _ = ref.backward(gu.bf16_bits(ybits), c.W, c.targets, c.ignore_index, 1.0, glp, None)
    seen = x64 if checkpoint is None else ops.rounded(x64, checkpoint)
    want = ops.layer_norm_grad(dy, seen, mean, rstd, ou.np64(w))
    for name, got, r in zip(("dx", "dweight", "dbias"), (x.grad, w.grad, b.grad), want):
        assert got.dtype == torch.float32
        assert gu.rel_max(ou.np64(got), r) <= gu.GRAD_RTOL, name
    assert lp.shape == (M,) and float(lp.detach().max()) <= 0


@pytest.mark.parametrize("checkpoint", [None, "mxint8"])
def test_layer_norm_autograd(checkpoint):
    """Three axes, an expanded gradient, parameters that need none."""
    import torch
    from log_prob_amd import autograd, flce
    x, w, b = norm_case(24, 136, 5, "bfloat16")
    x = x.view(2, 3, 4, 136).requires_grad_()
    w = w.bfloat16().requires_grad_()
    y = autograd.layer_norm(x, w, b.bfloat16(), EPS, checkpoint=checkpoint)
    assert y.shape == x.shape and y.dtype == torch.bfloat16
    y.sum().backward()   # the gradient is one element, expanded
    rows = x.detach().view(-1, 136)
    _, mean, rstd, *kept = flce.layer_norm_forward(rows, w, b.bfloat16(), EPS, checkpoint=checkpoint)
    dx, dw, _ = flce.layer_norm_backward(torch.ones_like(rows), kept[0] if kept else rows, mean, rstd, w)
    assert torch.equal(x.grad.view(-1, 136), dx) and torch.equal(w.grad, dw)
    # without parameters, and with a bias alone
    z = autograd.layer_norm(x, None, None, EPS, checkpoint=checkpoint)
    z.float().square().sum().backward()
    bias = b.bfloat16().requires_grad_()
    autograd.layer_norm(x.detach(), None, bias, EPS, checkpoint=checkpoint).sum().backward()
    assert bias.grad.dtype == torch.bfloat16 and (bias.grad == 24).all()


def test_layer_norm_gradient_against_differences():
    """The gradient along random directions against central differences of the fp64 norm."""
    import torch
    from log_prob_amd import autograd
    x, w, b = norm_case(5, 40, 6)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(5, 40, generator=gen, device="cuda")
    args = [v.requires_grad_() for v in (x, w, b)]
    (autograd.layer_norm(*args, EPS) * dy).sum().backward()
    f = lambda *a: float((ops.layer_norm(*a, EPS)[0] * ou.np64(dy)).sum())
    rng = np.random.default_rng(2)
    base = [ou.np64(v) for v in args]
    h = 1e-5
    for k, v in enumerate(args):
        d = rng.standard_normal(base[k].shape)
        lo, hi = list(base), list(base)
        lo[k], hi[k] = base[k] - h * d, base[k] + h * d
        want = (f(*hi) - f(*lo)) / (2 * h)
        got = float((ou.np64(v.grad) * d).sum())
        # fp32 gradients of about 40 roundings each; differences good to h^2
        scale = float(np.abs(ou.np64(v.grad) * d).sum())
        assert abs(got - want) <= 64 * ou.U32 * scale + 1e-7 * abs(want) + 1e-7


def test_scoring_and_sampling():
    """A step of a rollout: norm, then logits of the last token and log-probs of the batch with
    the 4-bit head, and the policy loss on them; the log-probs against the fp64 chain."""
    import torch
    from log_prob_amd import flce
    M, H, V = 300, 264, 1300
    x, w, b = norm_case(M, H, 7, "bfloat16")
    w, b = w.bfloat16(), b.bfloat16()
    gen = torch.Generator(device="cuda").manual_seed(8)
    W = flce.mx_quantize((torch.randn(V, H, generator=gen, device="cuda") / H ** 0.5).bfloat16(), "mxfp4")
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    y, _, _ = flce.layer_norm_forward(x, w, b, EPS)
    old, lse, _ = flce.mxfp4_forward(y, W, t)
    z = flce.mxfp4_logits(y, W, out_dtype=torch.float32)
    last = flce.mxfp4_logits(y[-1:].contiguous(), W, out_dtype=torch.float32)
    # one softmax, two ways to it: sums of 264 products in different orders
    Wv = ou.np64(flce.mx_dequantize(W, torch.float32))
    Xv = ops.rounded(ou.np64(y), "mxfp4")
    e = (H + 2) * 2 * ou.U32 * (np.abs(Xv) @ np.abs(Wv).T)
    assert (np.abs(ou.np64(last)[0] - ou.np64(z)[-1]) <= 2 * e[-1]).all()
    want = ops.fp4_forward(ou.np64(y), Wv, t.cpu().numpy())
    assert np.abs(ou.np64(old) - want["logprob"]).max() <= gu.FWD_ATOL
    assert np.abs(ou.np64(lse) - want["lse"]).max() <= gu.FWD_ATOL
    adv = torch.randn(M, generator=gen, device="cuda")
    per_tok, clipped, out = flce.policy_loss_reduce(old, old, adv, t, V)
    assert torch.equal(per_tok, -adv) and not clipped.any()   # the same policy: ratio 1


@pytest.mark.parametrize("M,H,V", [(6, 264, 1500), (40, 264, 1500), (300, 264, 1500),
                                   (500, 264, 32100), (4096, 256, 32800)],
                         ids=["own", "stream", "token_tiles", "tile", "queued_tiles"])
def test_graph_replays_match_eager(M, H, V):
    """A training step around the head and a pass of the 4-bit head in one captured graph,
    replayed with eager work and synchronisation between."""
    import torch
    from log_prob_amd import flce
    x, w, b = norm_case(M, H, 9)
    gen = torch.Generator(device="cuda").manual_seed(10)
    W = (torch.randn(V, H, generator=gen, device="cuda") / H ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    cb, sb = flce.mx_sizes(H, "mxint8")
    fb, sf = flce.mx_sizes(H, "mxfp4")
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    f32 = lambda *s: torch.empty(*s, device="cuda")
    y = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    kept = flce.MXTensor(u8(M, cb), u8(M, sb), "mxint8", H)
    Wq = flce.MXTensor(u8(V, fb), u8(V, sf), "mxfp4", H)
    mean, rstd, lp, lse, g = (f32(M) for _ in range(5))
    qlp, qlse, qent = (f32(M) for _ in range(3))
    red = torch.empty(3, dtype=torch.float64, device="cuda")
    dy, dW = torch.empty_like(y), torch.empty_like(W)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    z = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
    ws = u8(max(*flce.workspace_query(M, H, V, False), *flce.mxfp4_workspace_query(M, H, V),
                flce.layer_norm_backward_workspace(M, H)))
    outs = (y, kept.codes, kept.scales, Wq.codes, Wq.scales, mean, rstd, lp, lse, red, dy, dW, dx, dw,
            db, z, qlp, qlse, qent)

    def step():
        flce.layer_norm_forward(x, w, b, EPS, checkpoint="mxint8", out=(y, mean, rstd, kept))
        flce.forward(y, W, t, compute_entropy=False, workspace=ws, out=(lp, lse, None))
        flce.nll_reduce(lp, t, V, out=red)
        flce.nll_mean_grad(t, V, red, out=g)
        flce.backward(y, W, t, lse, None, g, workspace=ws, out=(dy, dW))
        flce.layer_norm_backward(dy, kept, mean, rstd, w, dx_dtype=x.dtype, workspace=ws, out=(dx, dw, db))
        flce.mx_quantize(W, "mxfp4", out=Wq)
        flce.mxfp4_logits(y, Wq, workspace=ws, out=z)
        flce.mxfp4_forward(y, Wq, t, workspace=ws, out=(qlp, qlse, qent))

    step()
    torch.cuda.synchronize()
    want = [v.clone() for v in outs]
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
        for v in outs:
            v.zero_()
        ws.fill_(0xFF)
        junk = (x @ x.T).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, r) in enumerate(zip(outs, want)):
            assert torch.equal(a, r), f"replay {i}: output {k} differs"
        del junk


@pytest.mark.parametrize("checkpoint", [None, "mxfp8"])
def test_captured_autograd_replays(checkpoint):
    """Forward and backward of the autograd norm in one captured graph, with no eager graph of
    its leaves alive; inputs changed between the replays."""
    import torch
    from log_prob_amd import autograd
    x, w, b = (v.requires_grad_() for v in norm_case(37, 264, 12))
    dy = torch.randn(37, 264, device="cuda")

    def step():
        y = autograd.layer_norm(x, w, b, EPS, checkpoint=checkpoint)
        return (y.detach(), *torch.autograd.grad(y, (x, w, b), dy))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        with torch.no_grad():
            x.add_(0.25)
            dy.mul_(-1.5)
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in outs]
        for a, r in zip(got, step()):
            assert torch.equal(a, r)


def test_two_streams_side_by_side():
    """The same calls on two streams at once, each with its own outputs and workspaces."""
    import torch
    from log_prob_amd import flce
    M, H, V = 600, 520, 3000
    sets = []
    for seed in (20, 21):
        x, w, b = norm_case(M, H, seed, "bfloat16")
        gen = torch.Generator(device="cuda").manual_seed(seed)
        W = flce.mx_quantize(torch.randn(V, H, generator=gen, device="cuda").bfloat16(), "mxfp4")
        sets.append((x, w.bfloat16(), b.bfloat16(), W, torch.randint(0, V, (M,), generator=gen, device="cuda")))

    def work(x, w, b, W, t):
        y, mean, rstd, kept = flce.layer_norm_forward(x, w, b, EPS, checkpoint="mxfp8")
        out = flce.mxfp4_forward(y, W, t)
        few = flce.mxfp4_logits(y[:9].contiguous(), W)
        return (y, few, *out, *flce.layer_norm_backward(y, kept, mean, rstd, w))

    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(work(*s))
        torch.cuda.synchronize()
        for g, r in zip(got, want):
            for a, e in zip(g, r):
                assert torch.equal(a, e)


def test_two_host_threads():
    """Two threads, each on a stream of its own, in calls that let go of the interpreter."""
    import threading
    import torch
    from log_prob_amd import flce
    jobs = []
    for seed, M, H, V in ((40, 3, 264, 5000), (41, 200, 520, 3000)):
        x, w, b = norm_case(M, H, seed, "bfloat16")
        gen = torch.Generator(device="cuda").manual_seed(seed)
        W = flce.mx_quantize(torch.randn(V, H, generator=gen, device="cuda"), "mxfp4")
        jobs.append((x, w.bfloat16(), b.bfloat16(), W, torch.randint(0, V, (M,), generator=gen, device="cuda")))

    def work(x, w, b, W, t):
        y, mean, rstd = flce.layer_norm_forward(x, w, b, EPS)
        return (y, flce.mxfp4_logits(y, W), *flce.mxfp4_forward(y, W, t),
                *flce.layer_norm_backward(y, x, mean, rstd, w))

    want = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def worker(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                runs = [work(*jobs[i]) for _ in range(30)]
            s.synchronize()
            got[i] = runs
        except Exception as err:   # reported by the test's thread
            errors.append(err)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for runs, ref_ in zip(got, want):
        for run in runs:
            assert all(torch.equal(a, r) for a, r in zip(run, ref_))


def test_plain_calls_and_given_buffers_agree():
    """The compiled binding of plain calls against the way that takes the results' buffers."""
    import torch
    from log_prob_amd import flce
    nat = flce._fast()
    gen = torch.Generator(device="cuda").manual_seed(30)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    f32 = lambda *s: torch.empty(*s, device="cuda")
    same = lambda a, b: all(torch.equal(u, v) and u.dtype == v.dtype for u, v in zip(a, b))
    for M, H, xd, yd, fmt in ((1, 264, "float32", "bfloat16", None), (7, 1000, "bfloat16", "bfloat16", "mxint8"),
                              (3, 33, "float32", "float32", "mxfp8"), (0, 64, "bfloat16", "bfloat16", None)):
        x, w, b = norm_case(max(M, 1), 2 * H, 31, xd)
        x, w, b = x[:M, :H], w[:H], b[:H]   # rows inside wider rows
        xd, yd = getattr(torch, xd), getattr(torch, yd)
        f = -1 if fmt is None else flce.MX_FORMATS[fmt]
        y, mean, rstd = torch.empty(M, H, dtype=yd, device="cuda"), f32(M), f32(M)
        kept = flce._mx_empty(M, H, fmt or "mxfp8", flce.MX_FORMATS[fmt or "mxfp8"], x.device)
        out = (y, mean, rstd) + ((kept,) if fmt else ())
        flce.layer_norm_forward(x, w, b, EPS, checkpoint=fmt, out=out)
        got = nat.layer_norm_forward(x, w, b, EPS, yd, f)
        assert got is not None and same(got, (y, mean, rstd) + ((kept.codes, kept.scales) if fmt else ()))
        dy = torch.randn(M, H, generator=gen, device="cuda").to(yd)
        src = kept if fmt else x
        dx, dw, db = torch.empty(M, H, dtype=xd, device="cuda"), f32(H), f32(H)
        flce.layer_norm_backward(dy, src, mean, rstd, w, dx_dtype=xd, out=(dx, dw, db))
        got = nat.layer_norm_backward(dy, None if fmt else x, kept.codes if fmt else None,
                                      kept.scales if fmt else None, f, mean, rstd, w, xd, True, None)
        assert got is not None and same(got, (dx, dw, db))
        got = nat.layer_norm_backward(dy, None if fmt else x, kept.codes if fmt else None,
                                      kept.scales if fmt else None, f, mean, rstd, w, xd, False, None)
        assert torch.equal(got[0], dx) and got[1] is None and got[2] is None
        for name, f in flce.MX_FORMATS.items():
            q = flce._mx_empty(M, H, name, f, x.device)
            flce.mx_quantize(x, name, out=q)
            assert same(nat.mx_quantize(x, f), (q.codes, q.scales))
            v = torch.empty(M, H, device="cuda")
            flce.mx_dequantize(q, out=v)
            assert torch.equal(nat.mx_dequantize(q.codes, q.scales, f, H, torch.float32), v)
    for M, H, V in ((1, 64, 100), (9, 264, 1300), (300, 72, 1001)):
        X = torch.randn(M, H, generator=gen, device="cuda").bfloat16()
        W = flce.mx_quantize(torch.randn(V, H, generator=gen, device="cuda"), "mxfp4")
        t = torch.randint(0, V, (M,), generator=gen, device="cuda")
        t[0] = -7
        z = torch.empty(M, V, dtype=torch.float32, device="cuda")
        flce.mxfp4_logits(X, W, 0.5, out=z)
        assert torch.equal(nat.mxfp4_logits(X, W.codes, W.scales, 0.5, torch.float32), z)
        out = (f32(M), f32(M), f32(M))
        flce.mxfp4_forward(X, W, t, -7, 0.5, out=out)
        assert same(nat.mxfp4_forward(X, W.codes, W.scales, t, -7, 0.5, True), out)
        got = nat.mxfp4_forward(X, W.codes, W.scales, t, -7, 0.5, False)
        assert same(got[:2], out[:2]) and got[2] is None


def test_compiled_binding_declines():
    """None, and nothing else, for what is not a plain valid call."""
    import torch
    from log_prob_amd import flce
    nat = flce._fast()
    x, w, b = norm_case(4, 64, 32)
    y, mean, rstd = flce.layer_norm_forward(x, w, b)
    q = flce.mx_quantize(x, "mxfp8")
    W = flce.mx_quantize(x, "mxfp4")
    X = x.bfloat16()
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    fwd = lambda *a: nat.layer_norm_forward(*a)
    ok = [x, w, b, EPS, None, -1]
    assert fwd(*ok) is not None
    for i, bad in ((0, x.half()), (0, x[0]), (0, x.t()), (0, x.cpu()), (0, x[0].expand(4, 64)), (0, None), (0, 3),
                   (1, w[:63]), (1, w.cpu()), (1, w.bfloat16()), (1, "w"), (2, b.half()), (2, b[::2]),
                   (3, "eps"), (3, -1.0), (3, float("nan")), (4, torch.float16), (4, 5), (5, 0), (5, "mxfp8")):
        a = list(ok)
        a[i] = bad
        assert fwd(*a) is None, (i, bad)
    assert fwd(*ok[:-1]) is None and fwd() is None
    assert fwd(X, None, None, EPS, torch.float32, -1) is None
    ok = [y, x, None, None, -1, mean, rstd, w, None, True, None]
    bwd = nat.layer_norm_backward
    assert bwd(*ok) is not None
    for i, bad in ((0, y[:3]), (0, y.cpu()), (1, x[:, :32]), (1, X), (1, None), (4, 1), (5, mean[:3]), (5, None),
                   (6, rstd.double()), (7, w[:5]), (8, torch.bfloat16), (8, torch.float16), (9, None),
                   (10, torch.bfloat16)):
        a = list(ok)
        a[i] = bad
        assert bwd(*a) is None, (i, bad)
    assert bwd(y, None, q.codes[:3], q.scales, 1, mean, rstd, w, None, True, None) is None
    assert bwd(y, None, q.codes, q.scales[:, :1], 1, mean, rstd, w, None, True, None) is None
    assert bwd(y, None, q.codes, q.scales, 0, mean, rstd, w, None, True, None) is None
    assert nat.mx_quantize(x.half(), 1) is None and nat.mx_quantize(x, 9) is None
    assert nat.mx_dequantize(q.codes, q.scales, 1, 65, None) is None
    assert nat.mx_dequantize(q.codes, q.scales, 1, 0, None) is None
    assert nat.mx_dequantize(q.codes, q.scales, 1, 1 << 70, None) is None
    assert nat.mxfp4_logits(x, W.codes, W.scales, 1.0, None) is None
    assert nat.mxfp4_logits(X[:, :32], W.codes, W.scales, 1.0, None) is None
    assert nat.mxfp4_logits(X, W.codes.cpu(), W.scales, 1.0, None) is None
    assert nat.mxfp4_logits(X, W.codes, W.scales, float("inf"), None) is None
    assert nat.mxfp4_forward(X, W.codes, W.scales, t.int(), -100, 1.0, True) is None
    assert nat.mxfp4_forward(X, W.codes, W.scales, t[:3], -100, 1.0, True) is None
    assert nat.mxfp4_forward(X, W.codes, W.scales, t, 1 << 70, 1.0, True) is None


def test_refusals():
    import torch
    from log_prob_amd import flce
    x, w, b = norm_case(4, 64, 11)
    y, mean, rstd = flce.layer_norm_forward(x, w, b)
    dy = torch.randn_like(y)
    with pytest.raises(TypeError):
        flce.layer_norm_forward(x.half(), w.half(), b.half())
    with pytest.raises(TypeError):
        flce.layer_norm_forward(x, w, b.bfloat16())
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x, w[:63], b)
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x, w[::2], b)
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x.t(), None, None)
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x[0].expand(4, 64), w, b)
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x.view(2, 2, 64), w, b)
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x, w, b, checkpoint="mxfp4")
    with pytest.raises(ValueError):
        flce.layer_norm_forward(x, w.cpu(), b)
    for bad in (lambda: flce.layer_norm_forward(x.bfloat16(), w, b, out_dtype=torch.float32),
                lambda: flce.layer_norm_forward(x, w, b, eps=-1.0),
                lambda: flce.layer_norm_backward(dy, x.bfloat16(), mean, rstd, w),
                lambda: flce.layer_norm_backward(dy, x, mean, rstd, w,
                                                 workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(flce.FlceError):
            bad()
    with pytest.raises(ValueError):
        flce.layer_norm_backward(dy, x[:3], mean, rstd, w)
    with pytest.raises(ValueError):
        flce.layer_norm_backward(dy, x, mean[:3], rstd, w)
    with pytest.raises(TypeError):
        flce.layer_norm_backward(dy, x, mean, rstd, w, dx_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        flce.layer_norm_backward(dy, flce.mx_quantize(x, "mxfp4"), mean, rstd, w)
    with pytest.raises(ValueError):
        flce.mx_dequantize(flce.mx_quantize(x, "mxfp8")._replace(cols=65))
    with pytest.raises(TypeError):
        flce.mx_dequantize(flce.mx_quantize(x, "mxfp8"), torch.float16)
    with pytest.raises(TypeError):
        flce.mx_quantize(x.half(), "mxfp8")
