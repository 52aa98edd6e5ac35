"""The residual block and log-probs from logits through the compiled binding and without it."""
import pytest

from log_prob_amd import flce


@pytest.mark.gpu
def test_the_same_results_without_the_binding(monkeypatch):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(60)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    X, W, b = n(40, 136).bfloat16(), n(520, 136).bfloat16(), n(520)
    r, dy, z = n(40, 520), n(40, 520).bfloat16(), n(40, 520)
    t = torch.randint(0, 520, (40, 3), generator=gen, device="cuda")
    seed = torch.tensor([-5], dtype=torch.int64, device="cuda")

    def flat(v):
        if torch.is_tensor(v):
            yield v
        elif isinstance(v, (tuple, list)):
            for e in v:
                yield from flat(e)

    def step():
        out = []
        for act in (None, "gelu"):
            y, pre = flce.linear_forward(X, W, b, act, r, torch.float32, keep_pre=True)
            out += [y, pre, flce.linear_forward(X[:3], W, None, act),
                    flce.linear_backward(dy, X, W, pre, act, bias_dtype=torch.bfloat16),
                    flce.linear_backward(dy, X, W, pre, act, need_dx=False)]
        out += [flce.dropout(dy, 0.3, 7, 9, r), flce.dropout(dy, 0.3, seed), flce.dropout_backward(r, 0.3, 7, 9, torch.bfloat16),
                flce.dropout(r, 0.25, (1 << 64) - 1, (1 << 64) - 1, out_dtype=torch.bfloat16)]
        for tok in (t, t[:, 0].contiguous(), None):
            for k in (0, 6):
                q = flce.token_logprobs(z, tok, scale=0.5, n_top=k, compute_entropy=k > 0)
                g = None if tok is None else torch.ones_like(q.logprob)
                out += [list(q), flce.token_logprobs_backward(z, tok, q.stats, q.entropy, q.top_ids, g,
                                                              q.top_logprob, q.entropy, q.lse, scale=0.5)]
        return list(flat(out))

    nat = flce._fast()
    assert not isinstance(nat, flce._Unbound)   # the tree that is tested has it
    # these calls are plain: the binding takes them
    assert nat.linear_forward(X, W, b, 2, r, torch.float32, True) is not None
    assert nat.linear_backward(dy, X, W, None, 0, True, True, None) is not None
    assert nat.dropout(dy, 0.3, 7, 9, r, None) is not None and nat.dropout(dy, 0.3, seed, 0, None, None) is not None
    assert nat.token_logprobs(z, t, -100, 1.0, 5, True) is not None
    want = step()
    monkeypatch.setattr(flce, "_native", flce._Unbound())
    got = step()
    assert len(got) == len(want) and all(torch.equal(a, e) for a, e in zip(got, want))


def test_the_binding_declines_host_tensors():
    import torch
    nat = flce._fast()
    x, X = torch.zeros(2, 32), torch.zeros(2, 32, dtype=torch.bfloat16)
    t = torch.zeros(2, dtype=torch.int64)
    assert nat.dropout(x, 0.1, 1, 0, None, None) is None
    assert nat.linear_forward(X, X, None, 0, None, None, False) is None
    assert nat.linear_backward(X, X, X, None, 0, True, True, None) is None
    assert nat.token_logprobs(x, t, -100, 1.0, 0, True) is None
    assert nat.token_logprobs_backward(x, t, x, None, None, None, None, None, None, -100, 1.0) is None
