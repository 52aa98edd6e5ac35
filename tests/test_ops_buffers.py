"""Workspaces a caller hands to the operators around the head: their bytes have to be there."""
import pytest

from log_prob_amd import flce


def test_workspace_bytes_must_exist():
    """A view that repeats or skips elements has more elements than bytes of its own from its
    first address on."""
    import torch
    dev = torch.device("cpu")
    ws = torch.zeros(4096, dtype=torch.uint8)
    assert flce._workspace(ws, 0, dev) is ws
    assert flce._workspace(ws[256:], 0, dev).numel() == 3840
    for bad in (ws[:1].expand(1 << 30), ws[::2], ws.view(64, 64).t(), ws.view(64, 64)[:, :8]):
        with pytest.raises(ValueError, match="contiguous"):
            flce._workspace(bad, 0, dev)
    with pytest.raises(ValueError, match="expected a tensor on"):
        flce._workspace(ws, 0, torch.device("cuda", 0))


@pytest.mark.gpu
def test_calls_refuse_a_repeated_workspace():
    import torch
    x = torch.randn(4, 64, device="cuda")
    X = x.bfloat16()
    W = flce.mx_quantize(torch.randn(300, 64, device="cuda"), "mxfp4")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    _, mean, rstd = flce.layer_norm_forward(x)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")[:1].expand(1 << 24)
    for call in (lambda: flce.layer_norm_backward(x, x, mean, rstd, workspace=ws),
                 lambda: flce.mxfp4_logits(X, W, workspace=ws),
                 lambda: flce.mxfp4_forward(X, W, t, workspace=ws)):
        with pytest.raises(ValueError, match="contiguous"):
            call()
