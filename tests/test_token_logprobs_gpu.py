"""Log-probs, entropy and alternatives from logits, and their gradient, on the GPU against the fp64
definition: ids exactly, values to bounds counted from the roundings (tests/block_util.py)."""
import numpy as np
import pytest

from oracle import block_ref as ref
from tests import block_util as bu
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def logits(M, V, dtype, seed, spread=3.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (spread * torch.randn(M, V, generator=gen, device="cuda")).to(dt(dtype))


def tokens(M, n, V, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000)
    t = torch.randint(0, V, (M, n), generator=gen, device="cuda")
    odd = torch.rand(M, n, generator=gen, device="cuda")
    t[odd < 0.05] = -100
    t[(odd > 0.05) & (odd < 0.08)] = V
    t[(odd > 0.08) & (odd < 0.1)] = -1
    return t


def check(x, t, n_top, scale=1.0, label="", entropy=True):
    """Against the definition; rows may be masked in part or throughout, not hold NaNs."""
    import torch
    from log_prob_amd import flce
    f32 = np.float32(scale)
    r = flce.token_logprobs(x, t, -100, float(f32), n_top, entropy)
    x64, t64 = ou.np64(x), t.cpu().numpy()
    t2 = t64.reshape(x.shape[0], -1)
    o = ref.token_logprobs(x64, t2, -100, float(f32), n_top)
    e_s, e_u = bu.sum_error(x64, float(f32), x.shape[1])
    with np.errstate(invalid="ignore"):
        d = float(f32) * (x64 - o["stats"][:, :1])
    logs = np.abs(o["stats"][:, 1])

    def close(got, want, bound, name):
        got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
        same = (got == want) | ~np.isfinite(want)
        assert np.array_equal(np.isfinite(got), np.isfinite(want)), f"{label} {name}"
        ou.check_within(np.where(same, 0, got), np.where(same, 0, want), np.broadcast_to(bound, got.shape), f"{label} {name}")
        assert np.array_equal(got[~np.isfinite(want)], want[~np.isfinite(want)]), f"{label} {name}"

    def at(ids):
        return np.nan_to_num(np.abs(np.take_along_axis(d, ids, 1)), nan=0, posinf=0)

    ok = ref.valid_tokens(t2, x.shape[1], -100)
    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0)
    close(ou.np64(r.logprob).reshape(t2.shape), o["logprob"],
          (e_s + 4 * ou.U32 * logs)[:, None] + 4 * ou.U32 * at(np.where(ok, t2, 0)) + ou.U32 * fin(o["logprob"]), "logprob")
    assert r.logprob.shape == t.shape
    close(ou.np64(r.lse), o["lse"], e_s + 4 * ou.U32 * (logs + fin(o["lse"]) + fin(o["stats"][:, 0]) * f32), "lse")
    close(ou.np64(r.stats[:, 0]), o["stats"][:, 0], 0, "largest logit")
    close(ou.np64(r.stats[:, 1]), o["stats"][:, 1], e_s + 4 * ou.U32 * logs, "log of the sum")
    if entropy:
        close(ou.np64(r.entropy), o["entropy"], e_s + e_u + 8 * ou.U32 * (logs + fin(o["entropy"])), "entropy")
    else:
        assert r.entropy is None
    if n_top:
        assert r.top_ids.dtype == torch.int64 and np.array_equal(r.top_ids.cpu().numpy(), o["top_ids"]), label
        close(ou.np64(r.top_logprob), o["top_logprob"],
              (e_s + 4 * ou.U32 * logs)[:, None] + 4 * ou.U32 * at(o["top_ids"]) + ou.U32 * fin(o["top_logprob"]), "top")
    else:
        assert r.top_ids is None and r.top_logprob is None
    return r, o


# one logit to many; pieces of a row of one vector and of several; whole and odd widths
SIZES = [(1, 1), (2, 2), (3, 7), (1, 8), (5, 64), (2, 255), (4, 1000), (1, 2048), (2, 2049), (1, 8192), (3, 8200),
         (2, 16391), (1, 50257), (2, 128256), (40, 20000), (300, 4097), (2100, 1032), (2050, 9001)]


@pytest.mark.parametrize("M,V", SIZES)
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_sizes(M, V, x):
    for n, k, scale in ((1, min(5, V), 1.0), (3, min(20, V), 1 / 0.7), (0, min(128, V), 0.25), (17, 0, 1.0)):
        check(logits(M, V, x, M + V), tokens(M, n, V, M + V), k, scale, f"{M}x{V} {x} n {n} k {k}", n != 3)


def test_one_token_a_row():
    x = logits(9, 777, "bf16", 3)
    check(x, tokens(9, 1, 777, 3)[:, 0].contiguous(), 4, label="1-d tokens")


@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [300, 9000, 70000])
@pytest.mark.parametrize("M", [1, 2060])
def test_orders_and_ties(V, x, M):
    """Rows that fill the candidates: ascending, descending, constant, two values, a saw of 2048, all
    of it in one thread's place; ties go to the lowest index."""
    import torch
    if M > 1 and V > 9000:
        M = 300
    i = torch.arange(V, device="cuda")
    rows = [i.float(), -i.float(), torch.full((V,), 1.5, device="cuda"), (i % 7 == 3).float(),
            (i % 2048).float(), ((i // 8) % 256 == 77).float() * i, torch.where(i == V - 1, 2.0, -1.0),
            torch.where(i % 2 == 0, 0.0, -0.0), (i // 1000).float()]
    z = torch.stack([rows[m % len(rows)] for m in range(max(M, len(rows)) if M > 1 else len(rows))]).to(dt(x))
    if x == "bf16":
        z = z.clamp(-30000, 30000)
    for part in ((z,) if M > 1 else z.split(1)):
        for k in (1, 20, 128):
            check(part, tokens(part.shape[0], 1, V, 5), k, 2.0 ** -10, f"order V {V} k {k}")


@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [64, 5000, 40000])
@pytest.mark.parametrize("M", [6, 2100])
def test_masks(V, x, M):
    """Masks of -inf and of the type's lowest value: in part, all but one, all but fewer than are
    asked for, throughout."""
    import torch
    if V == 40000 and M > 6:
        M = 60
    z = logits(M, V, x, 7)
    low = torch.finfo(z.dtype).min
    gen = torch.Generator(device="cuda").manual_seed(8)
    z[0::6][torch.rand(z[0::6].shape, generator=gen, device="cuda") < 0.9] = -float("inf")
    z[1::6, : V - 1] = -float("inf")
    z[2::6, 3:] = -float("inf")
    z[3::6] = -float("inf")
    z[4::6] = low
    z[5::6, : V // 2] = low
    t = tokens(M, 2, V, 9)
    t[:, 0] = V - 1
    for scale in (1.0, 0.5):
        check(z, t, min(30, V), scale, f"masks {V} {x}")
    r, _ = check(z, t, 5, 1.0, "masks")
    assert (r.lse[3::6] == -float("inf")).all() and (r.entropy[3::6] == 0).all()


@pytest.mark.parametrize("M", [4, 2100])
def test_rows_with_nan_or_infinity(M):
    import torch
    from log_prob_amd import flce
    V = 3001
    z = logits(M, V, "fp32", 10)
    clean = flce.token_logprobs(z, tokens(M, 2, V, 10), n_top=8)
    z[1, 5], z[1, 17], z[2, 2500] = float("nan"), float("inf"), float("inf")
    t = tokens(M, 2, V, 10)
    t[1, 0], t[1, 1] = 3, -100
    r = flce.token_logprobs(z, t, n_top=8)
    for m in (1, 2):
        assert torch.isnan(r.lse[m]) and torch.isnan(r.entropy[m]) and torch.isnan(r.top_logprob[m]).all()
        assert torch.isnan(r.stats[m]).all()
    assert torch.isnan(r.logprob[1, 0]) and r.logprob[1, 1] == 0
    o = ref.token_logprobs(ou.np64(z[1:3]), t[1:3].cpu().numpy(), n_top=8)
    assert np.array_equal(r.top_ids[1:3].cpu().numpy(), o["top_ids"])
    rest = [m for m in range(M) if m not in (1, 2)]
    for a, b in zip(r, clean):
        assert torch.equal(a[rest], b[rest])
    # and in the gradient
    g = torch.ones(M, 2, device="cuda")
    d = flce.token_logprobs_backward(z, t, r.stats, grad_logprob=g)
    assert torch.isnan(d[1:3]).all() and torch.isfinite(d[rest]).all()
    t[1] = -100   # nothing is asked of the row: no gradient
    assert (flce.token_logprobs_backward(z, t, r.stats, grad_logprob=g)[1] == 0).all()


def grad_check(x, t, r, k, scale, which, label):
    import torch
    from log_prob_amd import flce
    M, V = x.shape
    gen = torch.Generator(device="cuda").manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    t2 = t.reshape(M, -1)
    g = n(*t.shape) if "g" in which else None
    gt = n(M, k) if "t" in which else None
    ge = n(M) if "e" in which else None
    gl = n(M) if "l" in which else None
    got = flce.token_logprobs_backward(x, t, r.stats, r.entropy, r.top_ids, g, gt, ge, gl, -100, scale)
    assert got.dtype == x.dtype
    f = lambda a: None if a is None else ou.np64(a)
    ids = None if gt is None else r.top_ids.cpu().numpy()
    x64 = ou.np64(x)
    want = ref.token_logprobs_grad(x64, t2.cpu().numpy(), None if g is None else ou.np64(g).reshape(t2.shape), -100,
                                   scale, ids, f(gt), f(ge), f(gl))
    logp, d, logs, top, bad, none = ref._rows(x64, scale)
    p = np.exp(np.where(np.isfinite(logp), logp, -np.inf))
    lp = np.where(p > 0, np.abs(logp), 0)
    e_s, e_u = bu.sum_error(x64, scale, V)
    mag = sum(np.abs(f(a)).reshape(M, -1).sum(1) for a in (g, gt) if a is not None) if "g" in which or "t" in which else np.zeros(M)
    mag = mag + (0 if gl is None else np.abs(f(gl)))
    ent = np.abs(ref.token_logprobs(x64, t2.cpu().numpy(), -100, scale)["entropy"])
    b = np.zeros(M) if ge is None else np.abs(f(ge))
    # p from stored statistics, relative: theirs and the exponential's; then the coefficients
    rel = 2.0 ** -20 + e_s[:, None] + 6 * ou.U32 * (lp + np.abs(d) * (p > 0) + np.abs(logs)[:, None])
    rel = np.where(np.isfinite(rel), rel, 0)
    coef = mag[:, None] + b[:, None] * (lp + ent[:, None])
    e = scale * p * (coef * rel + b[:, None] * (rel + (e_s + e_u)[:, None]) + mag[:, None] * (t2.shape[1] + k + 8) * ou.U32)
    # the given tokens' own gradients, added in their order
    add = np.zeros((M, V))
    for tt, gg in ((t2.cpu().numpy(), None if g is None else ou.np64(g).reshape(t2.shape)), (ids, f(gt))):
        if gg is None:
            continue
        for m in range(M):
            for j in range(tt.shape[1]):
                if 0 <= tt[m, j] < V:
                    add[m, tt[m, j]] += abs(gg[m, j])
    e = e + scale * add * (t2.shape[1] + k + 4) * ou.U32
    ou.check_within(ou.np64(got), want, ou.half_step(x.dtype) * (np.abs(want) + e) + e, label)
    return got


@pytest.mark.parametrize("M,V", [(1, 1), (3, 7), (2, 64), (5, 1000), (1, 8192), (2, 8193), (3, 20011), (2, 50257), (300, 520)])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_gradient(M, V, x):
    for n, k, scale, which in ((1, 0, 1.0, "g"), (3, min(4, V), 0.5, "gtel"), (40, min(128, V), 1.0, "gt"),
                               (2, 0, 1.25, "e"), (1, 0, 1.0, "l")):
        z, t = logits(M, V, x, M + V), tokens(M, n, V, M + V)
        r, _ = check(z, t, k, scale)
        grad_check(z, t, r, k, scale, which, f"grad {M}x{V} {x} {n} {k} {which}")


def test_gradient_of_repeated_and_many_tokens():
    """One token several times, given and among the alternatives; a full list; the same bits again."""
    import torch
    V = 300
    z = logits(4, V, "fp32", 12)
    t = tokens(4, 1024, V, 13)   # each token of the row three times and more
    t[0, :] = 7
    r, _ = check(z, t, 128, 1.0)
    a = grad_check(z, t, r, 128, 1.0, "gte", "repeated")
    for _ in range(3):
        assert torch.equal(grad_check(z, t, r, 128, 1.0, "gte", "repeated"), a)


def test_gradient_under_masks():
    import torch
    z = logits(4, 2000, "bf16", 14)
    z[0, 100:] = -float("inf")
    z[1] = -float("inf")
    z[2] = torch.finfo(torch.bfloat16).min
    t = torch.tensor([[3, 50], [4, 5], [6, 1999], [-100, -100]], device="cuda")
    r, _ = check(z, t, 10, 1.0)
    d = grad_check(z, t, r, 10, 1.0, "ge", "masked")
    assert (d[0, 100:] == 0).all() and (d[1] == 0).all() and abs(float(d[2].float().sum())) < 1.0


@pytest.mark.parametrize("V,pad,shift", [(520, 8, 0), (520, 3, 1), (9001, 7, 2)])
def test_strides_and_in_place(V, pad, shift):
    import torch
    from log_prob_amd import flce
    M = 7
    z, t = logits(M, V, "bf16", 15), tokens(M, 5, V, 15)
    want = flce.token_logprobs(z, t, n_top=6)
    g = torch.randn(M, 5, device="cuda")
    dwant = flce.token_logprobs_backward(z, t, want.stats, want.entropy, grad_logprob=g, grad_entropy=g[:, 0].contiguous())
    buf = torch.full((M * (V + pad) + shift,), 9.0, dtype=z.dtype, device="cuda")
    view = buf[shift:].view(M, V + pad)[:, :V]
    view.copy_(z)
    out = flce.TokenLogprobs(*(torch.full_like(a, 3) for a in want))
    got = flce.token_logprobs(view, t, n_top=6, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(got, want))
    d = flce.token_logprobs_backward(view, t, want.stats, want.entropy, grad_logprob=g,
                                     grad_entropy=g[:, 0].contiguous(), out=view)
    assert d is view and torch.equal(view, dwant)
    assert (buf[shift:].view(M, V + pad)[:, V:] == 9).all() and (buf[:shift] == 9).all()


def test_offsets_past_32_bits():
    """17000 x 151936 logits (2.6e9, 5.2e9 bytes): the last rows as in a call of their own."""
    import gc
    import torch
    from log_prob_amd import flce
    M, V, n = 17000, 151936, 2100
    gen = torch.Generator(device="cuda").manual_seed(16)
    z = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
    for r in range(0, M, 1000):
        z[r:r + 1000] = torch.randn(1000, V, generator=gen, device="cuda")
    t = tokens(M, 2, V, 16)
    a = flce.token_logprobs(z, t, n_top=5)
    b = flce.token_logprobs(z[-n:].clone(), t[-n:].clone(), n_top=5)
    assert all(torch.equal(x[-n:], y) for x, y in zip(a, b))
    g = torch.randn(M, 2, device="cuda")
    want = flce.token_logprobs_backward(z[-n:].clone(), t[-n:].clone(), b.stats, grad_logprob=g[-n:].clone())
    flce.token_logprobs_backward(z, t, a.stats, grad_logprob=g, out=z)
    assert torch.equal(z[-n:], want)
    del z, want
    gc.collect()
    torch.cuda.empty_cache()


def test_empty_and_refusals():
    import torch
    from log_prob_amd import flce
    z, t = logits(4, 100, "fp32", 17), tokens(4, 2, 100, 17)
    e = flce.token_logprobs(z[:0], t[:0], n_top=3)
    assert e.logprob.shape == (0, 2) and e.top_ids.shape == (0, 3)
    assert flce.token_logprobs_backward(z[:0], t[:0], e.stats, grad_logprob=e.logprob).shape == (0, 100)
    r = flce.token_logprobs(z, t, n_top=3)
    for call in (lambda: flce.token_logprobs(z.half(), t), lambda: flce.token_logprobs(z, t.int()),
                 lambda: flce.token_logprobs_backward(z, t, r.stats.double()),
                 lambda: flce.token_logprobs_backward(z, t, r.stats, grad_logprob=r.logprob.bfloat16()),
                 lambda: flce.token_logprobs_backward(z, t, r.stats, grad_logprob=r.logprob, out=z.bfloat16())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: flce.token_logprobs(z[0], t), lambda: flce.token_logprobs(z, t[:3]),
                 lambda: flce.token_logprobs(z, t.t().contiguous().t()), lambda: flce.token_logprobs(z.t(), t),
                 lambda: flce.token_logprobs(z, t.cpu()), lambda: flce.token_logprobs_backward(z, t, r.stats[:3]),
                 lambda: flce.token_logprobs_backward(z, t, r.stats, grad_logprob=r.logprob[:, :1]),
                 lambda: flce.token_logprobs_backward(z, t, r.stats, grad_entropy=r.entropy),
                 lambda: flce.token_logprobs_backward(z, t, r.stats, grad_top=r.top_logprob),
                 lambda: flce.token_logprobs(z, t, n_top=2, out=r)):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(n_top=101), dict(n_top=-1),
               dict(n_top=129)):
        with pytest.raises(flce.FlceError):
            flce.token_logprobs(z, t, **kw)
