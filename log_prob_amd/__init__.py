"""libflce: fused LM-head linear + cross-entropy (log-prob, LSE, entropy) for gfx950, with
layer norm, microscaled formats and a head with 4-bit weights around it.

`log_prob_amd.flce` is the ctypes binding of the C ABI declared in include/flce.h;
`log_prob_amd.autograd` wraps it as torch.autograd.Functions (linear_logprob, layer_norm).
"""
__all__ = ["flce", "autograd"]
