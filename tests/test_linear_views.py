"""autograd.linear on views whose rows lie further apart than the matrix product takes (2^21 elements):
the last token of each sequence, every other row of a wide matrix."""
import pytest

LIMIT = 1 << 21   # row stride of X and W (include/flce.h)


@pytest.mark.parametrize("view", [lambda t: t[:, -1], lambda t: t[::2, 7], lambda t: t[1:, 3, :64]])
def test_operands_are_brought_within_the_limit(view):
    import torch
    from log_prob_amd.autograd import _as_operand
    x = view(torch.arange(4 * 1024 * 4096, dtype=torch.int32).view(4, 1024, 4096).bfloat16())
    assert x.stride(0) > LIMIT
    got = _as_operand(x, x.shape[-1])
    assert got.stride(0) <= LIMIT and got.stride(1) == 1 and got.stride(0) % 8 == 0 and torch.equal(got, x)


@pytest.mark.parametrize("D,rows", [(4096, 512), (4096, 513), (8, LIMIT // 8)])
def test_operands_within_it_are_not_copied(D, rows):
    import torch
    from log_prob_amd.autograd import _as_operand
    x = torch.zeros(2, rows, D, dtype=torch.bfloat16)[:, -1]
    assert (_as_operand(x, D).data_ptr() == x.data_ptr()) == (rows * D <= LIMIT)
    one = torch.zeros(1, 600, 4096, dtype=torch.bfloat16)[:, -1]   # a single row has no stride
    assert _as_operand(one, 4096).data_ptr() == one.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 4, 40])
def test_last_token_of_each_sequence(batch):
    import torch
    from log_prob_amd import autograd
    gen = torch.Generator(device="cuda").manual_seed(batch)
    h = torch.randn(batch, 520, 4096, generator=gen, device="cuda").bfloat16().requires_grad_()
    big = (torch.randn(48, 520, 4096, generator=gen, device="cuda") / 64).bfloat16()
    g = torch.randn(batch, 48, generator=gen, device="cuda").bfloat16()

    def run(x, w):
        w = w.detach().requires_grad_()
        y = autograd.linear(x, w, activation="silu")
        y.backward(g)
        return y.detach(), w.grad

    want = run(h[:, -1].contiguous(), big[:, 3].contiguous())
    dh, h.grad = h.grad, None
    got = run(h[:, -1], big[:, 3])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(h.grad, dh)
    assert (h.grad[:, :-1] == 0).all() and h.grad[:, -1].any()
