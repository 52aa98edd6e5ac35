"""The operators around the head without their compiled binding: the same calls through ctypes."""
import sys

import pytest

import log_prob_amd
from log_prob_amd import flce


@pytest.fixture
def unbound(monkeypatch, tmp_path):
    """No _binding.so to be found."""
    monkeypatch.delattr(log_prob_amd, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "log_prob_amd._binding", None)
    monkeypatch.setattr(flce, "_native", None)
    monkeypatch.setattr(flce, "HERE", str(tmp_path))
    return tmp_path


def test_calls_without_the_binding_still_check(unbound, recwarn):
    import torch
    x = torch.zeros(2, 32)
    for _ in range(2):
        with pytest.raises(ValueError, match="expected a GPU tensor"):
            flce.layer_norm_forward(x)
        with pytest.raises(ValueError, match="expected a GPU tensor"):
            flce.mx_quantize(x, "mxfp8")
    assert not recwarn.list


def test_a_binding_that_does_not_load_warns_once(unbound):
    import torch
    (unbound / "_binding.so").write_bytes(b"")
    with pytest.warns(RuntimeWarning, match="does not load"):
        with pytest.raises(ValueError):
            flce.mx_quantize(torch.zeros(2, 32), "mxfp8")
    import warnings
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError):
            flce.mx_quantize(torch.zeros(2, 32), "mxfp8")


@pytest.mark.gpu
def test_the_same_results_without_the_binding(monkeypatch):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(50)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, w, b, dy = n(9, 264), n(264), n(264), n(9, 264)
    t = torch.randint(0, 700, (9,), generator=gen, device="cuda")
    Wf = n(700, 264)

    def flat(r):
        if torch.is_tensor(r):
            yield r
        elif isinstance(r, (tuple, list)):
            for v in r:
                yield from flat(v)

    def step():
        y, mean, rstd, kept = flce.layer_norm_forward(x, w, b, out_dtype=torch.bfloat16, checkpoint="mxfp8")
        W = flce.mx_quantize(Wf, "mxfp4")
        return list(flat((y, mean, rstd, kept, W, flce.mx_dequantize(W),
                          flce.layer_norm_backward(dy, x, mean, rstd, w),
                          flce.layer_norm_backward(dy.bfloat16(), kept, mean, rstd, w, dx_dtype=torch.float32),
                          flce.mxfp4_logits(y, W, 0.5), flce.mxfp4_forward(y, W, t))))

    assert not isinstance(flce._fast(), flce._Unbound)   # the tree that is tested has it
    want = step()
    monkeypatch.setattr(flce, "_native", flce._Unbound())
    got = step()
    assert len(got) == len(want) and all(torch.equal(a, r) for a, r in zip(got, want))
