"""Operators on both sides of the LM head that are timed and compared: the residual block in
front of it, and the log-probs read off its logits.

  token_logprobs       log-probs of given tokens, log-sum-exp, entropy and the k largest logits
                       with their log-probs, from a matrix of logits
  token_logprobs_grad  the gradient of those log-probs and the entropy with respect to the logits
  linear               act(X W^T + bias) + residual, and the pre-activation where training keeps it
  linear_grad          dX, dW, dbias of it
  dropout              residual + dropout(x), and the gradient of x: a training step both ways

Log-probs are those of softmax(scale * logits).  A logit of -inf is masked: it has probability
0.  Alternatives are ordered by their logits, equal ones by their index.

Dropout drops an element where its 16 random bits are below round(65536 p), and divides what it
keeps by the probability that this leaves.  The bits come from Philox4x32-10 (Salmon, Moraes,
Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC11): the block with counter words
(column / 8, row, offset low, offset high) and key (seed low, seed high) serves the 8 columns
8 c .. 8 c + 7 of a row, two a word, the low half first.

With `own` false every operator runs in elementary torch operations in 32 bits; with `own`
true the same inputs go through log_prob_amd.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the sampler's answer for a small decode batch: latency
        dict(name="logprobs_decode", op="token_logprobs", M=4, V=128256, x="fp32", n=1, k=5, entropy=True, masked=0.0),
        # a constrained batch of a 50257-word vocabulary: half of each row masked, three tokens asked for
        dict(name="logprobs_masked_odd", op="token_logprobs", M=257, V=50257, x="fp32", n=3, k=8, entropy=True, masked=0.5),
        # scoring a batch of rollouts, the alternatives that a distillation keeps
        dict(name="logprobs_rollouts", op="token_logprobs", M=4096, V=128256, x="bf16", n=1, k=20, entropy=False, masked=0.0),
        # distillation: the log-probs of a teacher's 64 tokens a row
        dict(name="logprobs_grad_teacher", op="token_logprobs_grad", M=513, V=50257, x="fp32", n=64, entropy=False),
        # a policy's step with an entropy bonus
        dict(name="logprobs_grad_policy", op="token_logprobs_grad", M=4096, V=32768, x="bf16", n=1, entropy=True),
        # the residual block of a drafting head for one token: latency
        dict(name="linear_one_token", op="linear", M=1, N=4096, K=4096, act="silu", bias=True, residual="bf16", out="bf16", pre=False),
        # logits of a short ragged sequence over a 50257-word vocabulary
        dict(name="linear_logits_odd", op="linear", M=257, N=50257, K=1600, act="none", bias=False, residual="none", out="fp32", pre=False),
        # the dense block of a training batch
        dict(name="linear_batch", op="linear", M=4096, N=4096, K=4096, act="gelu", bias=True, residual="bf16", out="bf16", pre=True),
        # its gradient, for a short odd micro-batch and for the batch
        dict(name="linear_grad_odd", op="linear_grad", M=513, N=1000, K=2048, act="silu", bias=True, dy="fp32"),
        dict(name="linear_grad_batch", op="linear_grad", M=4096, N=4096, K=4096, act="gelu", bias=True, dy="bf16"),
        # a short odd micro-batch onto an fp32 residual stream: latency
        dict(name="dropout_short_odd", op="dropout", M=65, H=1000, x="bf16", residual="fp32", p=0.1),
        # a packed training batch
        dict(name="dropout_batch", op="dropout", M=32767, H=2048, x="bf16", residual="bf16", p=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["token_logprobs", "token_logprobs_grad", "linear", "linear_grad", "dropout"])
    if op == "dropout":
        H = _log_int(rng, 64, 8192)
        M = max(1, min(_log_int(rng, 1, 65536), 32767 * 2048 // H))
        x, r = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        return dict(op=op, M=M, H=H, x=x, residual=rng.choice([r, "none"]), p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    if op.startswith("linear"):
        M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 64, 50257), _log_int(rng, 64, 8192) // 8 * 8
        M = max(1, min(M, 4096**3 // (N * K), 4096 * 4096 // N))
        case = dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.7)
        if op == "linear_grad":
            return dict(case, dy=rng.choice(["bf16", "fp32"]))
        out = rng.choice(["bf16", "fp32"])
        return dict(case, residual=rng.choice(["none", out]), out=out, pre=case["act"] != "none" and rng.random() < 0.5)
    x = rng.choice(["bf16", "fp32"])
    V = _log_int(rng, 1000, 151936)
    most = 4096 * 128256 if op == "token_logprobs" else 4096 * 32768
    M = max(1, min(_log_int(rng, 1, 8192), most * 2 // (V * BYTES[x])))
    case = dict(op=op, M=M, V=V, x=x, n=rng.choice([1, 2, 5, 20, 64]), entropy=rng.random() < 0.5)
    if op == "token_logprobs":
        case.update(k=rng.choice([0, 1, 5, 20, 50]), masked=rng.choice([0.0, 0.5, 0.9]))
    return case


def work(case):
    op, M = case["op"], case["M"]
    if op == "dropout":
        n, x, r = M * case["H"], BYTES[case["x"]], BYTES.get(case["residual"], 0)
        y = r or x
        return {"bytes": n * (x + r + y) + n * (y + x), "flops": 30 * n}
    if op.startswith("linear"):
        N, K = case["N"], case["K"]
        operands = 2 * M * K + 2 * N * K
        if op == "linear":
            out = M * N * (BYTES[case["out"]] + BYTES.get(case["residual"], 0) + 2 * case["pre"])
            return {"bytes": operands + out + 4 * N * case["bias"], "flops": 2 * M * N * K}
        pre = 0 if case["act"] == "none" else 2 * M * N
        return {"bytes": 2 * operands + M * N * BYTES[case["dy"]] + pre + 4 * N * case["bias"], "flops": 4 * M * N * K}
    V, n, x = case["V"], case["n"], BYTES[case["x"]]
    if op == "token_logprobs":
        return {"bytes": M * V * x + 12 * M * n + 12 * M * case["k"] + 8 * M, "flops": 8 * M * V}
    return {"bytes": 2 * M * V * x + 12 * M * n + 8 * M, "flops": 8 * M * V}


# ---------------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _distinct(gen, M, n, V):
    """n tokens a row, no two alike."""
    first = torch.randint(0, V, (M, 1), generator=gen, device="cuda")
    return (first + torch.arange(n, device="cuda") * (V // n)) % V


def _logits(gen, case):
    """A head's logits: a broad spread, a few likely tokens a row; masked ones are -inf."""
    M, V = case["M"], case["V"]
    z = _normal(gen, M, V).mul_(2.0)
    likely = _distinct(gen, M, 12, V)
    z.scatter_(1, likely, 7.0 + 2.0 * _normal(gen, M, 12))
    masked = case.get("masked", 0.0)
    if masked:
        for r in range(0, M, 512):
            part = z[r : r + 512]
            gone = torch.rand(part.shape, generator=gen, device="cuda") < masked
            part.masked_fill_(gone.scatter_(1, likely[r : r + 512], False), -math.inf)
    return z.to(DTYPES[case["x"]]), likely


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    state = {"case": case}
    if op == "dropout":
        H = case["H"]
        state["x"] = _normal(gen, M, H).to(DTYPES[case["x"]])
        out = case["x"] if case["residual"] == "none" else case["residual"]
        state["residual"] = None if case["residual"] == "none" else (2.0 * _normal(gen, M, H)).to(DTYPES[out])
        state["dy"] = _normal(gen, M, H).to(DTYPES[out])
        state["seed"], state["offset"] = seed * 0x9E3779B97F4A7C15 % 2**64, seed
        return state
    if op.startswith("linear"):
        N, K = case["N"], case["K"]
        state["X"] = _normal(gen, M, K).to(torch.bfloat16)
        state["W"] = (_normal(gen, N, K) / math.sqrt(K)).to(torch.bfloat16)
        bias = (0.1 * _normal(gen, N)) if case["bias"] else None
        if op == "linear":
            state["bias"] = bias
            state["residual"] = None if case["residual"] == "none" else _normal(gen, M, N).to(DTYPES[case["out"]])
            return state
        state["dy"] = _normal(gen, M, N).to(DTYPES[case["dy"]])
        state["pre"] = None
        if case["act"] != "none":
            # what the forward kept
            pre = state["X"].float() @ state["W"].float().T
            state["pre"] = (pre if bias is None else pre + bias).to(torch.bfloat16)
        return state
    z, likely = _logits(gen, case)
    n, V = case["n"], case["V"]
    state["logits"] = z
    if n <= 12:
        tokens = likely[:, :n].clone()
    else:
        tokens = _distinct(gen, M, n, V)
    if not case.get("masked"):
        tokens = torch.where(torch.rand(M, n, generator=gen, device="cuda") < 0.05, IGNORE, tokens)
    state["tokens"] = tokens.contiguous()
    if op == "token_logprobs_grad":
        # what the forward kept: a row's largest logit, log of its sum, and its entropy
        stats, ent = torch.empty(M, 2, device="cuda"), torch.empty(M, device="cuda")
        for r in range(0, M, 512):
            part = z[r : r + 512].double()
            top = part.amax(1)
            d = part - top[:, None]
            ex = torch.exp(d)
            s = ex.sum(1)
            stats[r : r + 512, 0], stats[r : r + 512, 1] = top, torch.log(s)
            ent[r : r + 512] = torch.log(s) - (ex * d).sum(1) / s
        state["stats"], state["entropy"] = stats, ent
        state["grad_logprob"] = _normal(gen, M, n)
        state["grad_entropy"] = 0.1 * _normal(gen, M) if case["entropy"] else None
    return state


# ---------------------------------------------------------------------------- plain form
def _philox_bits(M, H, seed, offset, device):
    """16 random bits an element, as int32 [M, H]."""
    low = 0xFFFFFFFF
    blocks = -(-H // 8)
    c0 = torch.arange(blocks, device=device).expand(M, blocks)
    c1 = torch.arange(M, device=device)[:, None].expand(M, blocks)
    c2 = torch.full_like(c0, offset & low)
    c3 = torch.full_like(c0, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        # (64-bit products wrap around; their halves are taken as unsigned)
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), 2)
    return torch.stack((words & 0xFFFF, words >> 16), 3).view(M, blocks * 8)[:, :H].int()


def _plain_dropout(state):
    case, x, dy = state["case"], state["x"], state["dy"]
    t = int(round(65536 * case["p"]))
    keep = _philox_bits(*x.shape, state["seed"], state["offset"], x.device) >= t
    up = 65536 / (65536 - t)
    y = torch.where(keep, x.float() * up, 0.0)
    if state["residual"] is not None:
        y = state["residual"].float() + y
    return y.to(dy.dtype), torch.where(keep, dy.float() * up, 0.0).to(x.dtype)


def _act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_linear(state):
    case = state["case"]
    pre = state["X"].float() @ state["W"].float().T
    if state["bias"] is not None:
        pre = pre + state["bias"]
    y = _act(pre, case["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    y = y.to(DTYPES[case["out"]])
    return (y, pre.to(torch.bfloat16)) if case["pre"] else y


def _plain_linear_grad(state):
    case, g = state["case"], state["dy"].float()
    if case["act"] != "none":
        g = g * _act_slope(state["pre"].float(), case["act"])
    out = ((g @ state["W"].float()).to(torch.bfloat16), (g.T @ state["X"].float()).to(torch.bfloat16))
    return out + (g.sum(0),) if case["bias"] else out


def _plain_logprobs(state):
    case, z = state["case"], state["logits"].float()
    V, k, t = case["V"], case["k"], state["tokens"]
    top = z.amax(1, keepdim=True)
    d = z - top
    ex = torch.exp(d)
    s = ex.sum(1)
    logs = torch.log(s)
    here = d.gather(1, t.clamp(min=0)) - logs[:, None]
    out = (torch.where(t >= 0, here, 0.0), top[:, 0] + logs)
    if case["entropy"]:
        out += (logs - torch.where(ex > 0, ex * d, 0.0).sum(1) / s,)
    if k:
        # the bits of a float ordered as whole numbers, above the index from the end
        bits = (z + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2**18 + torch.arange(V - 1, -1, -1, device=z.device)
        ids = V - 1 - torch.topk(key, k, 1).values % 2**18
        out += (ids, d.gather(1, ids) - logs[:, None])
    return out


def _plain_logprobs_grad(state):
    z, t = state["logits"], state["tokens"]
    logp = z.float() - state["stats"][:, :1] - state["stats"][:, 1:]
    p = torch.exp(logp)
    g = torch.where(t >= 0, state["grad_logprob"], 0.0)
    dz = -g.sum(1, keepdim=True) * p
    if state["grad_entropy"] is not None:
        dz = dz - state["grad_entropy"][:, None] * p * (logp + state["entropy"][:, None])
    return dz.scatter_add_(1, t.clamp(min=0), g).to(z.dtype)


_PLAIN = {"token_logprobs": _plain_logprobs, "token_logprobs_grad": _plain_logprobs_grad, "linear": _plain_linear,
          "linear_grad": _plain_linear_grad, "dropout": _plain_dropout}


# ---------------------------------------------------------------------------- the framework's calls
def _calls(state):
    from log_prob_amd import flce
    case = state["case"]
    op = case["op"]
    act = None if case.get("act", "none") == "none" else case["act"]
    if op == "dropout":
        x, dy = state["x"], state["dy"]
        y = flce.dropout(x, case["p"], state["seed"], state["offset"], residual=state["residual"])
        return y, flce.dropout_backward(dy, case["p"], state["seed"], state["offset"], dx_dtype=x.dtype)
    if op == "linear":
        return flce.linear_forward(state["X"], state["W"], state["bias"], act, state["residual"],
                                   out_dtype=DTYPES[case["out"]], keep_pre=case["pre"])
    if op == "linear_grad":
        out = flce.linear_backward(state["dy"], state["X"], state["W"], state["pre"], act,
                                   bias_dtype=torch.float32 if case["bias"] else None)
        return out if case["bias"] else out[:2]
    if op == "token_logprobs":
        r = flce.token_logprobs(state["logits"], state["tokens"], IGNORE, n_top=case["k"], compute_entropy=case["entropy"])
        return ((r.logprob, r.lse) + ((r.entropy,) if case["entropy"] else ())
                + ((r.top_ids, r.top_logprob) if case["k"] else ()))
    return flce.token_logprobs_backward(state["logits"], state["tokens"], state["stats"], state["entropy"],
                                        grad_logprob=state["grad_logprob"], grad_entropy=state["grad_entropy"],
                                        ignore_index=IGNORE)


def run(state):
    return _calls(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64 bits
def _exact_words(M, H, seed, offset, device):
    """Philox4x32-10 in 16-bit limbs: [4, M, blocks]."""
    blocks = -(-H // 8)
    full = lambda v: torch.full((M, blocks), v, dtype=torch.int64, device=device)
    ctr = [torch.arange(blocks, device=device).repeat(M, 1), torch.arange(M, device=device)[:, None].repeat(1, blocks),
           full(offset % 2**32), full(offset // 2**32)]
    key = [seed % 2**32, seed // 2**32]

    def product(x, m):
        (xh, xl), (mh, ml) = (x // 65536, x % 65536), divmod(m, 65536)
        mid = xh * ml + (xl * ml) // 65536
        mid2 = xl * mh + mid % 65536
        return xh * mh + mid // 65536 + mid2 // 65536, mid2 % 65536 * 65536 + (xl * ml) % 65536

    for r in range(10):
        h0, l0 = product(ctr[0], 0xD2511F53)
        h1, l1 = product(ctr[2], 0xCD9E8D57)
        ks = [(key[0] + r * 0x9E3779B9) % 2**32, (key[1] + r * 0xBB67AE85) % 2**32]
        ctr = [h1.bitwise_xor(ctr[1]).bitwise_xor(full(ks[0])), l1, h0.bitwise_xor(ctr[3]).bitwise_xor(full(ks[1])), l0]
    return ctr


def _exact_dropout(state):
    case, x = state["case"], state["x"]
    M, H = x.shape
    drop = int(round(65536 * case["p"]))
    factor = torch.zeros(M, -(-H // 8) * 8, dtype=torch.float64, device=x.device)
    for w, word in enumerate(_exact_words(M, H, state["seed"], state["offset"], x.device)):
        factor[:, 2 * w :: 8] = torch.where(word % 65536 < drop, 0.0, 1 / (1 - drop / 65536))
        factor[:, 2 * w + 1 :: 8] = torch.where(word // 65536 < drop, 0.0, 1 / (1 - drop / 65536))
    factor = factor[:, :H]
    y = x.double() * factor
    return y if state["residual"] is None else y + state["residual"].double(), state["dy"].double() * factor


def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def _exact_act(z, name):
    """An activation and its slope."""
    if name == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if name == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z * z / 2) * 0.3989422804014327
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)
        s = torch.sigmoid(u2)
        return z * s, s + z * s * torch.sigmoid(-u2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z**2)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def _exact_linear(state):
    case = state["case"]
    X, W = state["X"].double(), state["W"].double()
    if case["op"] == "linear":
        pre = X @ W.t()
        if state["bias"] is not None:
            pre += state["bias"].double()
        y = _exact_act(pre, case["act"])[0]
        if state["residual"] is not None:
            y = y + state["residual"].double()
        return (y, pre) if case["pre"] else y
    g = state["dy"].double()
    if case["act"] != "none":
        g = g * _exact_act(state["pre"].double(), case["act"])[1]
    out = (g @ W, g.t() @ X)
    return out + (g.sum(0),) if case["bias"] else out


def _exact_logprobs(state):
    case, t = state["case"], state["tokens"]
    M, k = case["M"], case["k"]
    parts = []
    for r in range(0, M, 256):
        z, tr = state["logits"][r : r + 256].double(), t[r : r + 256]
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        part = [logp.gather(1, tr.clamp(min=0)).masked_fill(tr < 0, 0.0), lse]
        if case["entropy"]:
            part.append(-torch.nan_to_num(torch.exp(logp) * logp, nan=0.0).sum(1))
        if k:
            values, order = torch.sort(z, dim=1, descending=True, stable=True)
            part += [order[:, :k].clone(), values[:, :k] - lse[:, None]]
        parts.append(part)
    return tuple(torch.cat(p) for p in zip(*parts))


def _exact_logprobs_grad(state):
    case, t = state["case"], state["tokens"]
    out = torch.empty(case["M"], case["V"], dtype=torch.float64, device="cuda")
    for r in range(0, case["M"], 512):
        rows = slice(r, r + 512)
        logp = state["logits"][rows].double() - state["stats"][rows].double().sum(1, keepdim=True)
        p = torch.exp(logp)
        valid = t[rows] != IGNORE
        g = state["grad_logprob"][rows].double() * valid
        dz = -p * g.sum(1, keepdim=True)
        if state["grad_entropy"] is not None:
            # d(-sum p log p)/dz = -p (log p + H)
            dz -= state["grad_entropy"][rows].double()[:, None] * p * (logp + state["entropy"][rows].double()[:, None])
        row = torch.arange(p.shape[0], device="cuda")
        for j in range(case["n"]):
            dz[row, t[rows, j].clamp(min=0)] += g[:, j]
        out[rows] = dz
    return out


_EXACT = {"token_logprobs": _exact_logprobs, "token_logprobs_grad": _exact_logprobs_grad, "linear": _exact_linear,
          "linear_grad": _exact_linear, "dropout": _exact_dropout}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
