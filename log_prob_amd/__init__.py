"""libflce: fused LM-head linear + cross-entropy (log-prob, LSE, entropy) for gfx950, with
layer norm, microscaled formats, a head with 4-bit weights, a residual block (matrix product with
an epilogue, dropout) and log-probs from logits around it.

`log_prob_amd.flce` is the ctypes binding of the C ABI declared in include/flce.h;
`log_prob_amd.autograd` wraps it as torch.autograd.Functions (linear_logprob, layer_norm, linear,
dropout, token_logprobs).
"""
__all__ = ["flce", "autograd"]
