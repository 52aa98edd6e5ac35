"""Operators around the LM head that are timed and compared: layer norm in front of it,
8-bit checkpoints of the norm's input, and the head itself with 4-bit weights.

  norm_forward   y, mean, rstd of a layer norm over the last axis
  norm_backward  dx, dweight, dbias of it
  norm_saved8    the training step of a norm that keeps its input in 8 bits: the forward
                 writes y and the 8-bit copy, the backward reads the copy
  fp4_quantize   a matrix in microscaled 4-bit floating point, and the values it stands for
  fp4_logits     scale * Q(X) Wq^T for the sampler, W held in 4 bits
  fp4_logprob    log-prob, log-sum-exp and entropy of targets under those logits

Microscaled formats keep blocks of 32 consecutive elements of a row with one power-of-two
scale: the smallest 2^e (-127 <= e <= 127) at which no element of the block exceeds the
element format's largest value.  Elements are rounded to nearest, ties to even.  A scale
byte holds e + 127.  Formats: "mxfp4" (e2m1, two codes a byte, the even element in the low
half), "mxfp8" (e4m3) and "mxint8" (an integer in [-127, 127] over 64).  A row's codes are
padded with zeros to a whole block and its scale bytes to a multiple of 16.

With `own` false every operator runs in elementary torch operations in 32 bits; with `own`
true the same inputs go through log_prob_amd.
"""
import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token in a decode loop: latency
        dict(name="norm_forward_one_token", op="norm_forward", M=1, H=4096, x="bf16", y="bf16", p="bf16"),
        # a packed training batch, ragged token count
        dict(name="norm_forward_batch", op="norm_forward", M=32767, H=2048, x="bf16", y="bf16", p="bf16"),
        # an fp32 residual stream normalised into a bf16 head, fp32 parameters
        dict(name="norm_backward_mixed", op="norm_backward", M=4096, H=4096, x="fp32", y="bf16", p="fp32"),
        # the widest hidden size of the benchmark
        dict(name="norm_backward_wide", op="norm_backward", M=8192, H=8192, x="bf16", y="bf16", p="bf16"),
        # a short, odd micro-batch whose rows end inside a block of 32
        dict(name="norm_saved8_odd", op="norm_saved8", M=513, H=1000, x="fp32", y="fp32", p="fp32", fmt="mxfp8"),
        # a packed training batch with its checkpoint in integers
        dict(name="norm_saved8_batch", op="norm_saved8", M=32767, H=2048, x="bf16", y="bf16", p="bf16", fmt="mxint8"),
        # hidden states of a small decode batch
        dict(name="fp4_quantize_hidden", op="fp4_quantize", M=64, H=4096, x="bf16"),
        # a whole head, once per weight update of the policy
        dict(name="fp4_quantize_head", op="fp4_quantize", M=128256, H=4096, x="bf16"),
        # sampling one token from a 4-bit head
        dict(name="fp4_logits_one_token", op="fp4_logits", M=1, H=2048, V=151936, out="fp32"),
        # logits of a whole prompt
        dict(name="fp4_logits_prompt", op="fp4_logits", M=4096, H=4096, V=32768, out="bf16"),
        # scoring a short ragged sequence under a 50257-word vocabulary
        dict(name="fp4_logprob_short", op="fp4_logprob", M=257, H=1600, V=50257, entropy=True),
        # scoring a batch of rollouts with a frozen reference head
        dict(name="fp4_logprob_rollouts", op="fp4_logprob", M=4096, H=4096, V=128256, entropy=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "norm_saved8", "fp4_quantize", "fp4_logits", "fp4_logprob"])
    if op.startswith("norm") or op == "fp4_quantize":
        most = 8192 * 8192 if op != "fp4_quantize" else 128256 * 4096
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.75 or op == "norm_saved8":
            H = max(8, H // 8 * 8)
        M = max(1, min(_log_int(rng, 1, 131072 if op == "fp4_quantize" else 65536), most // H))
        if op == "fp4_quantize":
            return dict(op=op, M=M, H=H, x=rng.choice(["bf16", "fp32"]))
        x, y = rng.choice([("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
        case = dict(op=op, M=M, H=H, x=x, y=y, p=rng.choice(["fp32", y]))
        if op == "norm_saved8":
            case["fmt"] = rng.choice(["mxfp8", "mxint8"])
        return case
    H = _log_int(rng, 128, 8192) // 8 * 8
    V = _log_int(rng, 1000, 151936)
    most = 4096 * 4096 * (32768 if op == "fp4_logits" else 128256)
    M = _log_int(rng, 1, 8192)
    M = max(1, min(M, most // (H * V), 4096 * 128256 // V))
    if op == "fp4_logits":
        return dict(op=op, M=M, H=H, V=V, out=rng.choice(["bf16", "fp32"]))
    return dict(op=op, M=M, H=H, V=V, entropy=rng.random() < 0.5)


def work(case):
    op, M, H = case["op"], case["M"], case["H"]
    if op.startswith("norm"):
        x, y, p = BYTES[case["x"]], BYTES[case["y"]], BYTES[case["p"]]
        n = M * H
        fwd, bwd = n * (x + y) + 8 * M + 2 * H * p, n * (2 * x + y) + 8 * M + 3 * H * p
        if op == "norm_forward":
            return {"bytes": fwd, "flops": 8 * n}
        if op == "norm_backward":
            return {"bytes": bwd, "flops": 14 * n}
        saved = n + M * _scale_stride(H)
        return {"bytes": fwd + saved + n * (x + y) + saved + 8 * M + 3 * H * p, "flops": 26 * n}
    held = lambda rows: rows * (_blocks(H) * 16 + _scale_stride(H))
    if op == "fp4_quantize":
        # the matrix in, codes and scales out; codes and scales in, their values out
        return {"bytes": M * H * 2 * BYTES[case["x"]] + 2 * held(M), "flops": 4 * M * H}
    V = case["V"]
    bytes_ = 2 * M * H + held(V)
    bytes_ += M * V * BYTES[case["out"]] if op == "fp4_logits" else 8 * M + 12 * M
    return {"bytes": bytes_, "flops": 2 * M * H * V}


# ---------------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _hidden(gen, M, H):
    """A residual stream: unit normals around a small row offset, a few loud channels."""
    loud = torch.where(torch.rand(H, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return _normal(gen, M, H) * loud + 0.5 * _normal(gen, M, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, H = case["op"], case["M"], case["H"]
    state = {"case": case}
    if op.startswith("norm"):
        p = DTYPES[case["p"]]
        state["x"] = _hidden(gen, M, H).to(DTYPES[case["x"]])
        state["weight"] = (1.0 + 0.1 * _normal(gen, H)).to(p)
        state["bias"] = (0.1 * _normal(gen, H)).to(p)
        state["dy"] = _normal(gen, M, H).to(DTYPES[case["y"]])
        if op == "norm_backward":
            # what the forward kept
            x = state["x"].double()
            mean = x.mean(1)
            state["mean"] = mean.float()
            state["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS).float()
        return state
    if op == "fp4_quantize":
        state["x"] = (_hidden(gen, M, H) if M < 1024 else _normal(gen, M, H) / math.sqrt(H)).to(DTYPES[case["x"]])
        return state
    V = case["V"]
    state["X"] = _normal(gen, M, H).to(torch.bfloat16)
    e, codes = _mx_codes(_normal(gen, V, H) / math.sqrt(H), "mxfp4")
    state["w_codes"] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    state["w_scales"] = torch.zeros(V, _scale_stride(H), dtype=torch.uint8, device="cuda")
    state["w_scales"][:, : _blocks(H)] = (e + 127).to(torch.uint8)
    if op == "fp4_logprob":
        t = torch.randint(0, V, (M,), generator=gen, device="cuda")
        state["targets"] = torch.where(torch.rand(M, generator=gen, device="cuda") < 0.05, IGNORE, t)
    return state


# ---------------------------------------------------------------------------- plain form
def _blocks(H):
    return -(-H // 32)


def _scale_stride(H):
    return -(-_blocks(H) // 16) * 16


_MX = {"mxfp4": (2, 1.5, 6.0), "mxfp8": (8, 1.75, 448.0), "mxint8": (0, 127 / 64, 127 / 64)}


def _mx_blocks(x, fmt):
    """x as fp32 blocks [M, blocks, 32] over their scales, and the scales' exponents."""
    M, H = x.shape
    emax, mant, _ = _MX[fmt]
    v = torch.zeros(M, _blocks(H) * 32, dtype=torch.float32, device=x.device)
    v[:, :H] = x
    v = v.view(M, -1, 32)
    m, p = torch.frexp(v.abs().amax(2))
    e = torch.where(m > 0, p - 1 - emax + (2 * m > mant).int(), -127).clamp(-127, 127)
    return torch.ldexp(v, -e[:, :, None]), e


def _mx_codes(x, fmt):
    """Scale exponents [M, blocks] and e2m1 codes [M, 32 blocks] of a matrix."""
    assert fmt == "mxfp4"
    v, e = _mx_blocks(x, fmt)
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += (v < 0).to(torch.uint8) * 8
    return e, code.view(x.shape[0], -1)


def _mx_values(x, fmt):
    """The values that a matrix's microscaled copy stands for, in 32 bits."""
    M, H = x.shape
    v, e = _mx_blocks(x, fmt)
    if fmt == "mxint8":
        step = torch.full_like(v, 1 / 64)
    else:
        low, bits = (0, 1) if fmt == "mxfp4" else (-6, 3)
        step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 1).clamp(min=low) - bits)
    q = (torch.round(v / step) * step).clamp(-_MX[fmt][2], _MX[fmt][2])
    return torch.ldexp(q, e[:, :, None]).view(M, -1)[:, :H]


def _fp4_unpack(codes, scales, H):
    """The values of packed e2m1 codes and scale bytes, in 32 bits."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1)
    e = scales[:, : _blocks(H)].int() - 127
    v = grid[both.int()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, e[:, :, None]).view(codes.shape[0], -1)[:, :H]


def _plain_norm_forward(x, weight, bias, y_dtype):
    x = x.float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None] * weight.float() + bias.float()
    return y.to(y_dtype), mean, rstd


def _plain_norm_backward(dy, x, mean, rstd, weight, x_dtype):
    dy = dy.float()
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    g = dy * weight.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(x_dtype), (dy * xh).sum(0).to(weight.dtype), dy.sum(0).to(weight.dtype)


def _plain(state):
    case = state["case"]
    op, H = case["op"], case["H"]
    if op == "norm_forward":
        return _plain_norm_forward(state["x"], state["weight"], state["bias"], DTYPES[case["y"]])
    if op == "norm_backward":
        return _plain_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"], state["x"].dtype)
    if op == "norm_saved8":
        y, mean, rstd = _plain_norm_forward(state["x"], state["weight"], state["bias"], DTYPES[case["y"]])
        kept = _mx_values(state["x"].float(), case["fmt"])
        return (y, mean, rstd) + _plain_norm_backward(state["dy"], kept, mean, rstd, state["weight"], state["x"].dtype)
    if op == "fp4_quantize":
        return _mx_values(state["x"].float(), "mxfp4").to(state["x"].dtype)
    x = _mx_values(state["X"].float(), "mxfp4")
    z = x @ _fp4_unpack(state["w_codes"], state["w_scales"], H).T
    if op == "fp4_logits":
        return z.to(DTYPES[case["out"]])
    t = state["targets"]
    valid = t != IGNORE
    top = z.amax(1, keepdim=True)
    ex = torch.exp(z - top)
    s = ex.sum(1)
    lse = top[:, 0] + torch.log(s)
    zt = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    out = (torch.where(valid, zt - lse, 0.0), lse)
    if case["entropy"]:
        out += (torch.where(valid, torch.log(s) - (ex * (z - top)).sum(1) / s, 0.0),)
    return out


# ---------------------------------------------------------------------------- the framework's calls
def _calls(state):
    from log_prob_amd import flce
    case = state["case"]
    op, H = case["op"], case["H"]
    if op == "norm_forward":
        return flce.layer_norm_forward(state["x"], state["weight"], state["bias"], EPS, out_dtype=DTYPES[case["y"]])
    if op == "norm_backward":
        return flce.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])
    if op == "norm_saved8":
        y, mean, rstd, kept = flce.layer_norm_forward(state["x"], state["weight"], state["bias"], EPS, out_dtype=DTYPES[case["y"]],
                                                      checkpoint=case["fmt"])
        return (y, mean, rstd) + flce.layer_norm_backward(state["dy"], kept, mean, rstd, state["weight"], dx_dtype=state["x"].dtype)
    if op == "fp4_quantize":
        return flce.mx_dequantize(flce.mx_quantize(state["x"], "mxfp4"), state["x"].dtype)
    W = flce.MXTensor(state["w_codes"], state["w_scales"], "mxfp4", H)
    if op == "fp4_logits":
        return flce.mxfp4_logits(state["X"], W, out_dtype=DTYPES[case["out"]])
    lp, lse, ent = flce.mxfp4_forward(state["X"], W, state["targets"], IGNORE, compute_entropy=case["entropy"])
    return (lp, lse, ent) if case["entropy"] else (lp, lse)


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------- 64 bits
def _exact_grid(fmt):
    """Every non-negative value an element can take, in ascending order."""
    if fmt == "mxfp4":
        return [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    if fmt == "mxint8":
        return [k / 64 for k in range(128)]
    small = [k * 2.0**-9 for k in range(8)]
    return small + [(8 + k) * 2.0 ** (e - 3) for e in range(-6, 9) for k in range(8) if (e, k) != (8, 7)]


def _exact_values(x, fmt):
    """Microscaled values by search in the table of representable ones."""
    M, H = x.shape
    grid = torch.tensor(_exact_grid(fmt), dtype=torch.float64, device=x.device)
    out = torch.empty(M, H, dtype=torch.float64, device=x.device)
    rows = max(1, (1 << 26) // H)
    for r in range(0, M, rows):
        part = x[r : r + rows].double()
        n = part.shape[0]
        part = torch.nn.functional.pad(part, (0, _blocks(H) * 32 - H)).view(n, -1, 32)
        top = part.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2((top / grid[-1]).clamp(min=2.0**-127)))
        # log2 may round next to a whole number: settle it by comparison
        e = torch.where(top <= grid[-1] * torch.exp2(e - 1), e - 1, e)
        e = torch.where(top > grid[-1] * torch.exp2(e), e + 1, e).clamp(-127, 127)
        v = part.abs() / torch.exp2(e)
        hi = torch.searchsorted(grid, v.contiguous()).clamp(max=len(grid) - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - v, v - grid[lo]
        pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        q = grid[pick] * torch.exp2(e) * torch.sign(part)
        out[r : r + rows] = q.view(n, -1)[:, :H]
    return out


def _exact_norm(state, kept=None):
    x, w, dy = (state[k].double() for k in ("x", "weight", "dy"))
    H = x.shape[1]
    mean = x.sum(1) / H
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / H + EPS)
    y = w * ((x - mean[:, None]) * rstd[:, None]) + state["bias"].double()
    if "mean" in state:
        mean, rstd = state["mean"].double(), state["rstd"].double()
    xh = ((x if kept is None else kept) - mean[:, None]) * rstd[:, None]
    # dx as the Jacobian's product: (I - 11^T / H - xh xh^T / H) (w dy) rstd
    g = w * dy
    dx = (g - (g.sum(1) / H)[:, None] - xh * ((g * xh).sum(1) / H)[:, None]) * rstd[:, None]
    return y, mean, rstd, dx, (dy * xh).sum(0), dy.sum(0)


def exact(case, seed):
    state = prepare(case, seed)
    op, H = case["op"], case["H"]
    if op == "norm_forward":
        return _exact_norm(state)[:3]
    if op == "norm_backward":
        return _exact_norm(state)[3:]
    if op == "norm_saved8":
        return _exact_norm(state, _exact_values(state["x"], case["fmt"]))
    if op == "fp4_quantize":
        return _exact_values(state["x"], "mxfp4")
    X = _exact_values(state["X"], "mxfp4")
    table = torch.tensor(_exact_grid("mxfp4"), dtype=torch.float64, device="cuda")
    table = torch.cat((table, -table))
    z = torch.empty(case["M"], case["V"], dtype=torch.float64, device="cuda")
    for v in range(0, case["V"], 16384):
        c, s = state["w_codes"][v : v + 16384], state["w_scales"][v : v + 16384, : _blocks(H)]
        w = torch.empty(c.shape[0], 2 * c.shape[1], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = table[(c % 16).long()], table[(c // 16).long()]
        w *= torch.exp2(s.double() - 127).repeat_interleave(32, 1)
        z[:, v : v + 16384] = X @ w[:, :H].t()
    if op == "fp4_logits":
        return z
    t = state["targets"]
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    here = lp[torch.arange(case["M"], device="cuda"), t.clamp(min=0)]
    gone = t == IGNORE
    out = (here.masked_fill(gone, 0.0), lse)
    if case["entropy"]:
        out += (-(torch.exp(lp) * lp).sum(1).masked_fill(gone, 0.0),)
    return out
