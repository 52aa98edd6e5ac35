"""The residual block, the norm, a head's logits and the log-probs read off them as they are used
together: training steps by autograd and by hand, captured graphs, streams and host threads."""
import threading

import numpy as np
import pytest

from oracle import block_ref as ref
from oracle import ops_ref as ops
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

M, D, F, V = 70, 136, 264, 777
P, IGNORE = 0.2, -100


def weights(seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return dict(W1=(n(F, D) / D ** 0.5).bfloat16(), b1=0.1 * n(F), W2=(n(D, F) / F ** 0.5).bfloat16(), b2=0.1 * n(D),
                w=1 + 0.1 * n(D), b=0.1 * n(D), H=(n(V, D) / D ** 0.5).bfloat16())


def batch(seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + 500)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    t = torch.randint(0, V, (M, 2), generator=gen, device="cuda")
    t[torch.rand(M, 2, generator=gen, device="cuda") < 0.1] = IGNORE
    return dict(x=n(M, D).bfloat16(), t=t, g=n(M, 2), ge=0.1 * n(M), gl=0.1 * n(M), gt=0.1 * n(M, 4))


def forward(x, p, t, seed):
    """A dense block on a residual stream, the norm, and log-probs of the head's logits."""
    import torch
    from log_prob_amd import autograd as ag
    h = ag.linear(x, p["W1"], p["b1"], "gelu")
    y = ag.linear(h, p["W2"], p["b2"])
    r = ag.dropout(y, P, seed, 3, residual=x.float())
    u = ag.layer_norm(r, p["w"], p["b"], out_dtype=torch.bfloat16)
    z = ag.linear(u, p["H"], out_dtype=torch.float32)
    return ag.token_logprobs(z, t, IGNORE, 0.8, n_top=4, compute_entropy=True)


def step(s, p, seed):
    """Results and gradients by autograd."""
    import torch
    leaves = [s["x"].detach().requires_grad_()] + [v.detach().requires_grad_() for v in p.values()]
    q = forward(leaves[0], dict(zip(p, leaves[1:])), s["t"], seed)
    grads = torch.autograd.grad((q.logprob, q.entropy, q.lse, q.top_logprob), leaves, (s["g"], s["ge"], s["gl"], s["gt"]))
    return [v.detach() for v in q] + list(grads)


def by_hand(s, p, seed):
    """The same by the plain calls."""
    import torch
    from log_prob_amd import flce
    x = s["x"]
    h, pre = flce.linear_forward(x, p["W1"], p["b1"], "gelu", keep_pre=True)
    y = flce.linear_forward(h, p["W2"], p["b2"])
    r = flce.dropout(y, P, seed, 3, residual=x.float())
    u, mean, rstd = flce.layer_norm_forward(r, p["w"], p["b"], out_dtype=torch.bfloat16)
    z = flce.linear_forward(u, p["H"], out_dtype=torch.float32)
    q = flce.token_logprobs(z, s["t"], IGNORE, 0.8, 4)
    dz = flce.token_logprobs_backward(z, s["t"], q.stats, q.entropy, q.top_ids, s["g"], s["gt"], s["ge"], s["gl"], IGNORE, 0.8)
    du, dH, _ = flce.linear_backward(dz, u, p["H"])
    dr, dw, db = flce.layer_norm_backward(du, r, mean, rstd, p["w"])
    dy = flce.dropout_backward(dr, P, seed, 3, torch.bfloat16)
    dh, dW2, db2 = flce.linear_backward(dy, h, p["W2"], bias_dtype=torch.float32)
    dx, dW1, db1 = flce.linear_backward(dh, x, p["W1"], pre, "gelu", bias_dtype=torch.float32)
    return list(q) + [dx, dr.bfloat16(), dW1, db1, dW2, db2, dw, db, dH], (pre, h, y, r, mean, rstd, u, z, dz, du, dr, dy, dh)


def test_autograd_makes_the_plain_calls():
    import torch
    p, s = weights(1), batch(1)
    got = step(s, p, 17)
    want, _ = by_hand(s, p, 17)
    for a, b in zip(got[:6], want[:6]):
        assert torch.equal(a, b)
    # x's gradient: the block's and the residual's, added in bf16 by torch in either order
    assert torch.equal(got[6], want[6] + want[7])
    for a, b in zip(got[7:], want[8:]):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_chain_against_the_definitions():
    """Every stage from the values that the stage before it gave, in fp64, and the gradients back."""
    import torch
    p, s = weights(2), batch(2)
    out, (pre, h, y, r, mean, rstd, u, z, dz, du, dr, dy, dh) = by_hand(s, p, 99)
    f = ou.np64
    from tests import block_util as bu
    want, pre64, e, ep = bu.linear_bounds(f(s["x"]), f(p["W1"]), f(p["b1"]), "gelu", None, ou.U16)
    ou.check_within(f(h), want, e, "h")
    want, _, e, _ = bu.linear_bounds(f(h), f(p["W2"]), f(p["b2"]), None, None, ou.U16)
    ou.check_within(f(y), want, e, "y")
    want = ref.dropout(f(y), P, 99, 3, f(s["x"]))
    ou.check_within(f(r), want, 4 * ou.U32 * (np.abs(want) + 2 * np.abs(f(y))), "r")
    want, _, e, _ = bu.linear_bounds(f(u), f(p["H"]), None, None, None, ou.U32)
    ou.check_within(f(z), want, e, "z")
    o = ref.token_logprobs(f(z), s["t"].cpu().numpy(), IGNORE, float(np.float32(0.8)), 4)
    assert np.array_equal(out[3].cpu().numpy(), o["top_ids"])
    assert np.abs(f(out[0]) - o["logprob"]).max() <= 1e-5
    d = ref.token_logprobs_grad(f(z), s["t"].cpu().numpy(), f(s["g"]), IGNORE, float(np.float32(0.8)), o["top_ids"],
                                f(s["gt"]), f(s["ge"]), f(s["gl"]))
    assert np.abs(f(dz) - d).max() <= 2e-5 * np.abs(d).max()
    (wx, ex), (ww, ew), _ = bu.linear_grad_bounds(f(dz), f(u), f(p["H"]), None, None, True)
    ou.check_within(f(du), wx, ex, "du")
    ou.check_within(f(out[-1]), ww, ew, "dH")
    keep = ref.dropout_bits(M, D, 99, 3) >= round(65536 * P)
    assert np.array_equal(f(dy) != 0, keep & (f(dr) != 0))
    (wx, ex), (ww, ew), (wb, eb) = bu.linear_grad_bounds(f(dh), f(s["x"]), f(p["W1"]), f(pre), "gelu", True)
    for name, got, w, e in (("dx", out[6], wx, ex), ("dW1", out[8], ww, ew), ("db1", out[9], wb, eb)):
        ou.check_within(f(got), w, e, name)


def test_captured_training_step():
    """Forward and backward in a graph, replayed over new inputs, weights and seeds, with eager work
    between; the seed lives in device memory."""
    import torch
    p = weights(3)
    s = batch(3)
    seed = torch.tensor([5], dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s, p, seed)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s, p, seed)
    for k in range(4):
        for a, b in zip(s.values(), batch(10 + k).values()):
            a.copy_(b)
        for a, b in zip(p.values(), weights(20 + k).values()):
            a.copy_(b)
        seed.fill_(1000 + k)
        graph.replay()
        held = [v.clone() for v in got]
        torch.cuda.synchronize()
        want = step(s, p, 1000 + k)
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_captured_decoding_step():
    """One token through the block and the head, and its alternatives (pieces of a row, split K)."""
    import torch
    from log_prob_amd import flce
    n = lambda *q: torch.randn(*q, device="cuda")
    W, b, H = (n(2048, 2048) / 45).bfloat16(), n(2048), (n(50257, 2048) / 45).bfloat16()
    for m in (1, 16):
        x, t = n(m, 2048).bfloat16(), torch.randint(0, 50257, (m,), device="cuda")

        def decode():
            y = flce.linear_forward(x, W, b, "silu", residual=x)
            return flce.token_logprobs(flce.linear_forward(y, H, out_dtype=torch.float32), t, n_top=20)

        decode()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = decode()
        for k in range(3):
            x.copy_(n(m, 2048))
            t.copy_(torch.randint(0, 50257, (m,), device="cuda"))
            graph.replay()
            held = [v.clone() for v in got]
            assert all(torch.equal(a, c) for a, c in zip(held, decode()))


def test_two_graphs_do_not_share_a_workspace():
    """Two captured calls replayed at once on streams of their own."""
    import torch
    from log_prob_amd import flce
    cases, graphs = [], []
    for k in range(2):
        gen = torch.Generator(device="cuda").manual_seed(k)
        n = lambda *q: torch.randn(*q, generator=gen, device="cuda")
        cases.append((n(40, 4096).bfloat16(), (n(512, 4096) / 64).bfloat16(), n(3, 90000), torch.randint(0, 512, (40,), device="cuda")))

    def run(c):
        y = flce.linear_forward(c[0], c[1], out_dtype=torch.float32)
        a, b, _ = flce.linear_backward(y, c[0], c[1])
        return [y, a, b] + [v for v in flce.token_logprobs(c[2], None, n_top=9) if v is not None]

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(c)
        graphs.append((g, out))
    for _ in range(3):
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_two_streams_and_two_threads():
    import torch
    p, s = weights(5), [batch(6), batch(7)]
    want = [step(s[k], p, 40 + k) for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = step(s[k], p, 40 + k)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for k in range(2) for a, b in zip(got[k], want[k]))
    failed = []

    def work(k):
        try:
            with torch.cuda.stream(streams[k]):
                for _ in range(5):
                    got[k] = step(s[k], p, 40 + k)
                streams[k].synchronize()
        except Exception as err:   # noqa: BLE001
            failed.append(err)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert all(torch.equal(a, b) for k in range(2) for a, b in zip(got[k], want[k]))


def test_autograd_shapes_views_and_what_needs_no_gradient():
    import torch
    from log_prob_amd import autograd as ag
    n = lambda *q: torch.randn(*q, device="cuda")
    x = n(2, 3, 64).bfloat16().requires_grad_()
    W, b = (n(48, 64) / 8).bfloat16().requires_grad_(), n(48).requires_grad_()
    r = n(2, 3, 48).requires_grad_()
    y = ag.linear(x, W, b, "silu", r, torch.float32)
    z = ag.dropout(y, 0.5, 3, residual=r)
    assert y.shape == z.shape == (2, 3, 48) and z.dtype == torch.float32
    z.sum().backward()   # an expanded gradient
    flat = ag.linear(x.detach().reshape(6, 64), W, b, "silu", r.detach().reshape(6, 48), torch.float32)
    assert torch.equal(flat, y.detach().view(6, 48))
    keep = torch.from_numpy(ref.dropout_bits(6, 48, 3, 0) >= 32768).cuda().view(2, 3, 48)
    assert torch.equal(r.grad, 1 + 2.0 * keep)
    assert x.grad.shape == x.shape and W.grad.shape == W.shape and b.grad.shape == b.shape
    # operands that are views with rows that are not aligned, or not contiguous
    wide = n(6, 131).bfloat16()
    for v in (wide[:, 3:67], wide[:, :64], wide.t()[:64].t()):
        assert torch.equal(ag.linear(v, W), ag.linear(v.contiguous(), W))
    # only some need a gradient
    only = ag.linear(x.detach(), W.detach(), b, "relu")
    g, = torch.autograd.grad(only.float().sum(), b)
    assert torch.equal(g, (ag.linear(x.detach(), W.detach(), b) > 0).float().sum((0, 1)))
    none = ag.linear(x.detach(), W.detach(), None, "relu")
    assert not none.requires_grad
    logits = n(5, 40).requires_grad_()
    q = ag.token_logprobs(logits, None, n_top=3)
    assert q.entropy is None and q.logprob.shape == (5, 0) and not q.top_ids.requires_grad and not q.stats.requires_grad
    q.top_logprob.sum().backward()
    want, = torch.autograd.grad(torch.log_softmax(logits.double(), 1).gather(1, q.top_ids).sum(), logits)
    assert torch.allclose(logits.grad.double(), want.double(), atol=1e-5)
    for bad in (lambda: ag.linear(x, W, residual=r[0]), lambda: ag.dropout(x, 0.1, 1, residual=x[0])):
        with pytest.raises(ValueError):
            bad()


def test_dropout_seed_tensor_changed_before_the_backward():
    """The graph keeps the seed that the forward drew with."""
    import torch
    from log_prob_amd import autograd as ag
    x = torch.ones(9, 72, device="cuda", requires_grad=True)
    seed = torch.tensor([11], dtype=torch.int64, device="cuda")
    y = ag.dropout(x, 0.5, seed)
    seed.fill_(12)
    y.sum().backward()
    assert torch.equal(x.grad, y.detach()) and not torch.equal(ag.dropout(x, 0.5, seed).detach(), y.detach())
