"""Thin ctypes binding of libflce (the C ABI in include/flce.h).

Only argument marshalling lives here: every step of the computation runs in the
HIP kernels of libflce.so.  torch supplies device memory and the current stream.
If the library is missing, loading fails loudly; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Any, NamedTuple, Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libflce.so")

FLCE_OK = 0
# bytes of the static device scratch flce_forward_noalloc uses (FLCE_NOALLOC_SCRATCH_BYTES)
FLCE_NOALLOC_SCRATCH_BYTES = 32 << 20
STATUS = {0: "FLCE_OK", 1: "FLCE_ERR_INVALID_VALUE", 2: "FLCE_ERR_UNSUPPORTED",
          3: "FLCE_ERR_WORKSPACE_TOO_SMALL", 4: "FLCE_ERR_HIP"}

# Every symbol include/flce.h declares.
EXPORTS = ("flce_workspace_query", "flce_forward_workspace_min", "flce_forward_wave_rows",
           "flce_backward_workspace_min", "flce_backward_chunk_cols",
           "flce_backward_wave_rows", "flce_backward_schedule", "flce_forward",
           "flce_forward_noalloc", "flce_forward_partials", "flce_forward_merge", "flce_backward",
           "flce_forward_partials_shard", "flce_forward_merge_shards",
           "flce_backward_shard_workspace_query", "flce_backward_shard", "flce_nll_reduce",
           "flce_nll_mean_grad", "flce_policy_loss_reduce", "flce_policy_loss_grad",
           "flce_mx_sizes", "flce_mx_quantize", "flce_mx_dequantize", "flce_layer_norm_forward",
           "flce_layer_norm_backward_workspace", "flce_layer_norm_backward",
           "flce_mx_workspace_query", "flce_mx_logits", "flce_mx_forward",
           "flce_linear_workspace", "flce_linear_forward", "flce_linear_backward", "flce_dropout",
           "flce_token_logprobs_workspace", "flce_token_logprobs", "flce_token_logprobs_backward",
           "flce_status_string",
           "flce_last_error_message", "flce_version")

_lib = None


class FlceError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libflce.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libflce.so not built at {path}; run `python -m log_prob_amd.build`")
    try:
        # torch brings a HIP runtime of its own: loaded first, it is the one that libflce.so binds to
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    c = ctypes
    P, I64, SZ = c.c_void_p, c.c_int64, c.c_size_t
    lib.flce_workspace_query.argtypes = [I64, I64, I64, c.c_int, c.POINTER(SZ), c.POINTER(SZ)]
    lib.flce_forward_workspace_min.argtypes = [I64, I64, I64, c.c_int, c.POINTER(SZ)]
    lib.flce_forward_wave_rows.argtypes = [I64, I64, I64, c.c_int, SZ, c.POINTER(I64)]
    lib.flce_backward_workspace_min.argtypes = [I64, I64, I64, c.POINTER(SZ)]
    lib.flce_backward_chunk_cols.argtypes = [I64, I64, I64, SZ, c.POINTER(I64)]
    lib.flce_backward_wave_rows.argtypes = [I64, I64, I64, SZ, c.POINTER(I64)]
    lib.flce_backward_schedule.argtypes = [I64, I64, I64, SZ, c.POINTER(I64), c.POINTER(I64),
                                           c.POINTER(c.c_int)]
    lib.flce_forward.argtypes = [P, P, P, I64, I64, I64, I64, c.c_float, c.c_int, P, P, P, P, SZ, P]
    lib.flce_forward_noalloc.argtypes = [P, P, P, I64, I64, I64, I64, c.c_float, c.c_int, P, P, P,
                                         P]
    lib.flce_forward_partials.argtypes = [P, P, P, I64, I64, I64, I64, c.c_float, c.c_int, P, SZ,
                                          P]
    lib.flce_forward_merge.argtypes = [P, I64, I64, I64, I64, c.c_int, P, P, P, P, SZ, P]
    lib.flce_backward.argtypes = [P, P, P, I64, I64, I64, I64, c.c_float, P, P, P, P, P, P, P,
                                  SZ, P]
    lib.flce_forward_partials_shard.argtypes = [P, P, P, I64, I64, I64, I64, I64, c.c_float,
                                                c.c_int, P, SZ, P]
    lib.flce_forward_merge_shards.argtypes = [P, I64, I64, c.POINTER(I64), I64, c.c_int, P, P, P,
                                              P, SZ, P]
    lib.flce_backward_shard_workspace_query.argtypes = [I64, I64, I64, c.POINTER(SZ),
                                                        c.POINTER(SZ)]
    lib.flce_backward_shard.argtypes = [P, P, P, I64, I64, I64, I64, I64, I64, c.c_float, P, P, P,
                                        P, P, c.c_int, P, P, SZ, P]
    lib.flce_nll_reduce.argtypes = [P, P, I64, I64, I64, P, P]
    lib.flce_nll_mean_grad.argtypes = [P, I64, I64, I64, P, P, P]
    D = c.c_double
    lib.flce_policy_loss_reduce.argtypes = [P, P, P, P, I64, I64, I64, D, D, D, P, P, P, P]
    lib.flce_policy_loss_grad.argtypes = [P, P, P, P, I64, I64, I64, D, D, D, P, P, P]
    I = c.c_int
    lib.flce_mx_sizes.argtypes = [I64, I, c.POINTER(I64), c.POINTER(I64)]
    lib.flce_mx_quantize.argtypes = [P, I, I64, I64, I64, I, P, P, P]
    lib.flce_mx_dequantize.argtypes = [P, P, I, I64, I64, P, I, I64, P]
    lib.flce_layer_norm_forward.argtypes = [P, I, I64, P, P, I, I64, I64, c.c_float, P, I, I64, P,
                                            P, I, P, P, P]
    lib.flce_layer_norm_backward_workspace.argtypes = [I64, I64, c.POINTER(SZ)]
    lib.flce_layer_norm_backward.argtypes = [P, I, I64, P, I, I64, I, P, P, P, I, P, P, I64, I64,
                                             P, I, I64, P, P, P, SZ, P]
    lib.flce_mx_workspace_query.argtypes = [I64, I64, I64, I, c.POINTER(SZ), c.POINTER(SZ)]
    lib.flce_mx_logits.argtypes = [P, P, P, I64, I64, I64, c.c_float, P, I, I64, P, SZ, P]
    lib.flce_mx_forward.argtypes = [P, P, P, P, I64, I64, I64, I64, c.c_float, I, P, P, P, P, SZ, P]
    U64, F = c.c_uint64, c.c_float
    lib.flce_linear_workspace.argtypes = [I64, I64, I64, c.POINTER(SZ), c.POINTER(SZ)]
    lib.flce_linear_forward.argtypes = [P, I64, P, I64, P, I, I, P, I, I64, I64, I64, I64, P, I,
                                        I64, P, I64, P, SZ, P]
    lib.flce_linear_backward.argtypes = [P, I, I64, P, I64, I, P, I64, P, I64, I64, I64, I64, P,
                                         I64, P, I64, P, I, P, SZ, P]
    lib.flce_dropout.argtypes = [P, I, I64, P, I, I64, I64, I64, D, U64, P, U64, P, I, I64, P]
    lib.flce_token_logprobs_workspace.argtypes = [I64, I64, I64, c.POINTER(SZ)]
    lib.flce_token_logprobs.argtypes = [P, I, I64, I64, I64, P, I64, I64, F, I64, P, P, P, P, P, P,
                                        P, SZ, P]
    lib.flce_token_logprobs_backward.argtypes = [P, I, I64, I64, I64, P, I64, I64, F, P, P, P, I64,
                                                 P, P, P, P, P, I64, P]
    for name in ("flce_linear_workspace", "flce_linear_forward", "flce_linear_backward",
                 "flce_dropout", "flce_token_logprobs_workspace", "flce_token_logprobs",
                 "flce_token_logprobs_backward", "flce_mx_workspace_query", "flce_mx_logits", "flce_mx_forward",
                 "flce_mx_sizes", "flce_mx_quantize", "flce_mx_dequantize",
                 "flce_layer_norm_forward", "flce_layer_norm_backward_workspace",
                 "flce_layer_norm_backward", "flce_nll_reduce", "flce_nll_mean_grad",
                 "flce_policy_loss_reduce", "flce_policy_loss_grad", "flce_workspace_query",
                 "flce_forward_workspace_min", "flce_forward_wave_rows",
                 "flce_backward_workspace_min", "flce_backward_chunk_cols",
                 "flce_backward_wave_rows", "flce_backward_schedule", "flce_forward",
           "flce_forward_noalloc", "flce_forward_partials", "flce_forward_merge", "flce_backward",
                 "flce_forward_partials_shard", "flce_forward_merge_shards",
                 "flce_backward_shard_workspace_query", "flce_backward_shard"):
        getattr(lib, name).restype = c.c_int
    lib.flce_status_string.argtypes = [c.c_int]
    lib.flce_status_string.restype = c.c_char_p
    lib.flce_last_error_message.argtypes = []
    lib.flce_last_error_message.restype = c.c_char_p
    lib.flce_version.argtypes = []
    lib.flce_version.restype = c.c_char_p
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != FLCE_OK:
        raise FlceError(status, load().flce_last_error_message().decode())


def workspace_query(M: int, H: int, V: int, compute_entropy: bool = True) -> Tuple[int, int]:
    fwd, bwd = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().flce_workspace_query(M, H, V, int(bool(compute_entropy)), ctypes.byref(fwd),
                                       ctypes.byref(bwd)))
    return fwd.value, bwd.value


def forward_workspace_min(M: int, H: int, V: int, compute_entropy: bool = True) -> int:
    b = ctypes.c_size_t()
    _check(load().flce_forward_workspace_min(M, H, V, int(bool(compute_entropy)), ctypes.byref(b)))
    return b.value


def forward_wave_rows(M: int, H: int, V: int, workspace_bytes: int,
                      compute_entropy: bool = True) -> int:
    r = ctypes.c_int64()
    _check(load().flce_forward_wave_rows(M, H, V, int(bool(compute_entropy)), workspace_bytes,
                                         ctypes.byref(r)))
    return r.value


def backward_workspace_min(M: int, H: int, V: int) -> int:
    b = ctypes.c_size_t()
    _check(load().flce_backward_workspace_min(M, H, V, ctypes.byref(b)))
    return b.value


def backward_chunk_cols(M: int, H: int, V: int, workspace_bytes: int) -> int:
    c = ctypes.c_int64()
    _check(load().flce_backward_chunk_cols(M, H, V, workspace_bytes, ctypes.byref(c)))
    return c.value


def backward_wave_rows(M: int, H: int, V: int, workspace_bytes: int) -> int:
    r = ctypes.c_int64()
    _check(load().flce_backward_wave_rows(M, H, V, workspace_bytes, ctypes.byref(r)))
    return r.value


def backward_schedule(M: int, H: int, V: int, workspace_bytes: int):
    """(rows per token wave, chunk columns, pipelined) of flce_backward's schedule."""
    r, cc, pp = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
    _check(load().flce_backward_schedule(M, H, V, workspace_bytes, ctypes.byref(r),
                                         ctypes.byref(cc), ctypes.byref(pp)))
    return r.value, cc.value, bool(pp.value)


def backward_shard_workspace_query(M: int, H: int, V_shard: int) -> Tuple[int, int]:
    lo, pref = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().flce_backward_shard_workspace_query(M, H, V_shard, ctypes.byref(lo),
                                                      ctypes.byref(pref)))
    return lo.value, pref.value


# ----------------------------------------------------------------------------
# torch-facing wrappers
def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require(t, name, dtype, shape):
    import torch
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: expected a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def alloc_workspace(nbytes: int, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def forward(X, W, targets, ignore_index: int = -100, scale: float = 1.0,
            compute_entropy: bool = True, workspace=None, out=None):
    """(logprob, lse, entropy-or-None) as fp32 [M] tensors, on X's device and stream."""
    import torch
    M, H = X.shape
    V = W.shape[0]
    _require(X, "X", torch.bfloat16, (M, H))
    _require(W, "W", torch.bfloat16, (V, H))
    _require(targets, "targets", torch.int64, (M,))
    dev = X.device
    if out is None:
        logprob = torch.empty(M, dtype=torch.float32, device=dev)
        lse = torch.empty(M, dtype=torch.float32, device=dev)
        entropy = torch.empty(M, dtype=torch.float32, device=dev) if compute_entropy else None
    else:
        logprob, lse, entropy = out
    if workspace is None:
        fwd_b, _ = workspace_query(M, H, V, compute_entropy)
        workspace = alloc_workspace(fwd_b, dev)
    _check(load().flce_forward(_ptr(X), _ptr(W), _ptr(targets), M, H, V, int(ignore_index),
                               float(scale), int(bool(compute_entropy)), _ptr(logprob), _ptr(lse),
                               _ptr(entropy), _ptr(workspace), workspace.numel(), _stream(dev)))
    return logprob, lse, entropy


def forward_noalloc(X, W, targets, ignore_index: int = -100, scale: float = 1.0,
                    compute_entropy: bool = True, out=None):
    """flce_forward_noalloc: the forward through the library's static device scratch (no
    workspace).  With `out` = (logprob, lse, entropy-or-None) nothing is allocated here
    either; calls overlapping on one GPU share the scratch and must not run concurrently."""
    import torch
    M, H = X.shape
    V = W.shape[0]
    _require(X, "X", torch.bfloat16, (M, H))
    _require(W, "W", torch.bfloat16, (V, H))
    _require(targets, "targets", torch.int64, (M,))
    dev = X.device
    if out is None:
        logprob = torch.empty(M, dtype=torch.float32, device=dev)
        lse = torch.empty(M, dtype=torch.float32, device=dev)
        entropy = torch.empty(M, dtype=torch.float32, device=dev) if compute_entropy else None
    else:
        logprob, lse, entropy = out
    _check(load().flce_forward_noalloc(_ptr(X), _ptr(W), _ptr(targets), M, H, V,
                                       int(ignore_index), float(scale),
                                       int(bool(compute_entropy)), _ptr(logprob), _ptr(lse),
                                       _ptr(entropy), _stream(dev)))
    return logprob, lse, entropy


def forward_partials(X, W, targets, ignore_index: int = -100, scale: float = 1.0,
                     compute_entropy: bool = True, workspace=None):
    """Run only the fused GEMM + online-softmax kernel; partials stay in `workspace`."""
    import torch
    M, H = X.shape
    V = W.shape[0]
    _require(X, "X", torch.bfloat16, (M, H))
    _require(W, "W", torch.bfloat16, (V, H))
    _require(targets, "targets", torch.int64, (M,))
    if workspace is None:
        workspace = alloc_workspace(workspace_query(M, H, V, compute_entropy)[0], X.device)
    _check(load().flce_forward_partials(_ptr(X), _ptr(W), _ptr(targets), M, H, V,
                                        int(ignore_index), float(scale),
                                        int(bool(compute_entropy)), _ptr(workspace),
                                        workspace.numel(), _stream(X.device)))
    return workspace


def forward_merge(targets, M: int, H: int, V: int, workspace, ignore_index: int = -100,
                  compute_entropy: bool = True, out=None):
    """Merge partials left by forward_partials into (logprob, lse, entropy-or-None)."""
    import torch
    _require(targets, "targets", torch.int64, (M,))
    dev = targets.device
    if out is None:
        logprob = torch.empty(M, dtype=torch.float32, device=dev)
        lse = torch.empty(M, dtype=torch.float32, device=dev)
        entropy = torch.empty(M, dtype=torch.float32, device=dev) if compute_entropy else None
    else:
        logprob, lse, entropy = out
    _check(load().flce_forward_merge(_ptr(targets), M, H, V, int(ignore_index),
                                     int(bool(compute_entropy)), _ptr(logprob), _ptr(lse),
                                     _ptr(entropy), _ptr(workspace), workspace.numel(),
                                     _stream(dev)))
    return logprob, lse, entropy


def backward(X, W, targets, lse, entropy=None, grad_logprob=None, grad_entropy=None,
             ignore_index: int = -100, scale: float = 1.0, workspace=None, out=None):
    """(dX, dW) as bf16 tensors shaped like X and W."""
    import torch
    M, H = X.shape
    V = W.shape[0]
    _require(X, "X", torch.bfloat16, (M, H))
    _require(W, "W", torch.bfloat16, (V, H))
    _require(targets, "targets", torch.int64, (M,))
    _require(lse, "lse", torch.float32, (M,))
    for name, t in (("entropy", entropy), ("grad_logprob", grad_logprob),
                    ("grad_entropy", grad_entropy)):
        if t is not None:
            _require(t, name, torch.float32, (M,))
    dev = X.device
    if out is None:
        dX = torch.empty_like(X)
        dW = torch.empty_like(W)
    else:
        dX, dW = out
    if workspace is None:
        _, bwd_b = workspace_query(M, H, V, entropy is not None)
        workspace = alloc_workspace(bwd_b, dev)
    _check(load().flce_backward(_ptr(X), _ptr(W), _ptr(targets), M, H, V, int(ignore_index),
                                float(scale), _ptr(lse), _ptr(entropy), _ptr(grad_logprob),
                                _ptr(grad_entropy), _ptr(dX), _ptr(dW), _ptr(workspace),
                                workspace.numel(), _stream(dev)))
    return dX, dW


# ----------------------------------------------------------------------------
# vocabulary shards: what one rank of a vocabulary-parallel group runs
def forward_partials_shard(X, W_shard, targets, v_offset: int, ignore_index: int = -100,
                           scale: float = 1.0, compute_entropy: bool = True, workspace=None):
    """Partials of the shard W_shard = rows [v_offset, v_offset + V_shard) of W."""
    import torch
    M, H = X.shape
    Vs = W_shard.shape[0]
    _require(X, "X", torch.bfloat16, (M, H))
    _require(W_shard, "W_shard", torch.bfloat16, (Vs, H))
    _require(targets, "targets", torch.int64, (M,))
    if workspace is None:
        workspace = alloc_workspace(workspace_query(M, H, Vs, compute_entropy)[0], X.device)
    _check(load().flce_forward_partials_shard(_ptr(X), _ptr(W_shard), _ptr(targets), M, H, Vs,
                                              int(v_offset), int(ignore_index), float(scale),
                                              int(bool(compute_entropy)), _ptr(workspace),
                                              workspace.numel(), _stream(X.device)))
    return workspace


def forward_merge_shards(targets, shard_offsets, gathered, shard_stride_bytes: int,
                         ignore_index: int = -100, compute_entropy: bool = True, out=None):
    """Merge gathered shard partials (shard r at byte r * stride of `gathered`)."""
    import torch
    M = targets.shape[0]
    _require(targets, "targets", torch.int64, (M,))
    offs = (ctypes.c_int64 * len(shard_offsets))(*[int(v) for v in shard_offsets])
    dev = targets.device
    if out is None:
        logprob = torch.empty(M, dtype=torch.float32, device=dev)
        lse = torch.empty(M, dtype=torch.float32, device=dev)
        entropy = torch.empty(M, dtype=torch.float32, device=dev) if compute_entropy else None
    else:
        logprob, lse, entropy = out
    _check(load().flce_forward_merge_shards(_ptr(targets), M, len(shard_offsets) - 1, offs,
                                            int(ignore_index), int(bool(compute_entropy)),
                                            _ptr(logprob), _ptr(lse), _ptr(entropy),
                                            _ptr(gathered), int(shard_stride_bytes),
                                            _stream(dev)))
    return logprob, lse, entropy


def backward_shard(X, W_shard, targets, v_offset: int, V_total: int, lse, entropy=None,
                   grad_logprob=None, grad_entropy=None, dX_partial=None, accumulate=False,
                   ignore_index: int = -100, scale: float = 1.0, workspace=None, dW_shard=None):
    """(dX_partial fp32 [M, H], dW_shard bf16) of one shard; dX is the sum over shards."""
    import torch
    M, H = X.shape
    Vs = W_shard.shape[0]
    _require(X, "X", torch.bfloat16, (M, H))
    _require(W_shard, "W_shard", torch.bfloat16, (Vs, H))
    _require(targets, "targets", torch.int64, (M,))
    _require(lse, "lse", torch.float32, (M,))
    for name, t in (("entropy", entropy), ("grad_logprob", grad_logprob),
                    ("grad_entropy", grad_entropy)):
        if t is not None:
            _require(t, name, torch.float32, (M,))
    dev = X.device
    if dX_partial is None:
        dX_partial = torch.empty((M, H), dtype=torch.float32, device=dev)
    _require(dX_partial, "dX_partial", torch.float32, (M, H))
    if dW_shard is None:
        dW_shard = torch.empty_like(W_shard)
    if workspace is None:
        workspace = alloc_workspace(backward_shard_workspace_query(M, H, Vs)[1], dev)
    _check(load().flce_backward_shard(_ptr(X), _ptr(W_shard), _ptr(targets), M, H, Vs,
                                      int(v_offset), int(V_total), int(ignore_index),
                                      float(scale), _ptr(lse), _ptr(entropy),
                                      _ptr(grad_logprob), _ptr(grad_entropy), _ptr(dX_partial),
                                      int(bool(accumulate)), _ptr(dW_shard), _ptr(workspace),
                                      workspace.numel(), _stream(dev)))
    return dX_partial, dW_shard


# ----------------------------------------------------------------------------
# scalar cross-entropy reductions on the log-probs
def nll_reduce(logprob, targets, V: int, ignore_index: int = -100, out=None):
    """fp64 device tensor [sum of -logprob over valid rows, valid rows, mean NLL]."""
    import torch
    M = logprob.shape[0]
    _require(logprob, "logprob", torch.float32, (M,))
    _require(targets, "targets", torch.int64, (M,))
    if out is None:
        out = torch.empty(3, dtype=torch.float64, device=logprob.device)
    _require(out, "out", torch.float64, (3,))
    _check(load().flce_nll_reduce(_ptr(logprob), _ptr(targets), M, int(V), int(ignore_index),
                                  _ptr(out), _stream(logprob.device)))
    return out


def nll_mean_grad(targets, V: int, reduced, ignore_index: int = -100, out=None):
    """grad_logprob of the mean NLL (-1/n on valid rows) from nll_reduce's output."""
    import torch
    M = targets.shape[0]
    _require(targets, "targets", torch.int64, (M,))
    _require(reduced, "reduced", torch.float64, (3,))
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=targets.device)
    _require(out, "grad_logprob", torch.float32, (M,))
    _check(load().flce_nll_mean_grad(_ptr(targets), M, int(V), int(ignore_index), _ptr(reduced),
                                     _ptr(out), _stream(targets.device)))
    return out


def _policy_inputs(logprob, old_logprob, advantages, targets):
    import torch
    M = logprob.shape[0]
    _require(logprob, "logprob", torch.float32, (M,))
    if old_logprob is not None:
        _require(old_logprob, "old_logprob", torch.float32, (M,))
    _require(advantages, "advantages", torch.float32, (M,))
    _require(targets, "targets", torch.int64, (M,))
    return M


def policy_loss_reduce(logprob, old_logprob, advantages, targets, V: int,
                       ignore_index: int = -100, eps_low: float = 0.2, eps_high: float = 0.2,
                       denominator: float = 0.0, with_clip_flags: bool = True, out=None):
    """Clipped policy loss on the log-probs, token-mean aggregated (see include/flce.h):
    (per-token loss fp32 [M], clip flags uint8 [M] or None, fp64 device tensor [loss sum,
    valid rows, clipped rows, loss sum / N]).  `out` may supply those three buffers."""
    import torch
    M = _policy_inputs(logprob, old_logprob, advantages, targets)
    dev = logprob.device
    if out is not None:
        per_token, clipped, out = out
    else:
        per_token = torch.empty(M, dtype=torch.float32, device=dev)
        clipped = torch.empty(M, dtype=torch.uint8, device=dev) if with_clip_flags else None
        out = torch.empty(4, dtype=torch.float64, device=dev)
    _require(per_token, "per_token_loss", torch.float32, (M,))
    if clipped is not None:
        _require(clipped, "is_clipped", torch.uint8, (M,))
    _require(out, "out", torch.float64, (4,))
    _check(load().flce_policy_loss_reduce(
        _ptr(logprob), _ptr(old_logprob), _ptr(advantages), _ptr(targets), M, int(V),
        int(ignore_index), float(eps_low), float(eps_high), float(denominator), _ptr(per_token),
        _ptr(clipped), _ptr(out), _stream(dev)))
    return per_token, clipped, out


def policy_loss_grad(logprob, old_logprob, advantages, targets, V: int, reduced=None,
                     ignore_index: int = -100, eps_low: float = 0.2, eps_high: float = 0.2,
                     denominator: float = 0.0, out=None):
    """grad_logprob of the loss of policy_loss_reduce; `reduced` is its fp64 output
    (needed when denominator <= 0)."""
    import torch
    M = _policy_inputs(logprob, old_logprob, advantages, targets)
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=logprob.device)
    _require(out, "grad_logprob", torch.float32, (M,))
    if reduced is not None:
        _require(reduced, "reduced", torch.float64, (4,))
    _check(load().flce_policy_loss_grad(
        _ptr(logprob), _ptr(old_logprob), _ptr(advantages), _ptr(targets), M, int(V),
        int(ignore_index), float(eps_low), float(eps_high), float(denominator), _ptr(reduced),
        _ptr(out), _stream(logprob.device)))
    return out


# ----------------------------------------------------------------------------
# operators around the head: microscaled formats and the layer norm in front of it
MX_FORMATS = {"mxfp4": 0, "mxfp8": 1, "mxint8": 2}
_MX_NONE = -1


class MXTensor(NamedTuple):
    """A matrix [rows, cols] in a microscaled format: uint8 codes and scale bytes, laid out
    as include/flce.h states (mx_quantize makes them)."""
    codes: Any
    scales: Any
    fmt: str
    cols: int


class _Unbound:
    """Stands in for the compiled binding where it was not built: every call goes the long way."""

    def __getattr__(self, name):
        return lambda *args: None


_native = None


def _fast():
    """The compiled binding of the calls below (csrc/binding.cpp).  Its functions return None
    where a call is not plain and valid; what follows here then decides, or raises.  Without it
    every call takes that way, through ctypes into the same library, a few microseconds longer."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (the binding's libraries)
        load()
        try:
            from . import _binding
            _native = _binding
        except ImportError as err:
            if os.path.exists(os.path.join(HERE, "_binding.so")):
                import warnings
                warnings.warn(f"log_prob_amd/_binding.so does not load ({err}): calls go through "
                              "ctypes; `python -m log_prob_amd.build` makes one for this torch",
                              RuntimeWarning, stacklevel=3)
            _native = _Unbound()
    return _native


_DTYPE_IDS = {}   # torch dtype -> flce_dtype_t


def _dtype_id(t, name) -> int:
    d = _DTYPE_IDS.get(t.dtype)
    if d is None:
        import torch
        _DTYPE_IDS.update({torch.bfloat16: 0, torch.float32: 1})
        d = _DTYPE_IDS.get(t.dtype)
        if d is None:
            raise TypeError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return d


def _rows(t, name, dev, shape=None):
    """Check a matrix whose rows are contiguous; returns its row stride."""
    if t.device != dev:
        raise ValueError(f"{name}: expected a tensor on {dev}, got {t.device}")
    size = t.shape
    if len(size) != 2:
        raise ValueError(f"{name}: expected a matrix, got {len(size)} dimensions")
    if shape is not None and shape != size:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(size)}")
    m, h = size
    ld, one = t.stride()
    if one != 1 and h > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if m <= 1:
        return h
    if ld < h:
        raise ValueError(f"{name}: rows overlap")
    return ld


def _on_gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a GPU tensor")
    return t.device


def _vector(t, name, dev, dtype, n):
    if t.dtype == dtype and t.device == dev and t.shape == (n,) and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name}: expected a tensor on {dev}, got {t.device}")
    raise ValueError(f"{name}: expected {n} contiguous elements, got shape {tuple(t.shape)}")


def _workspace(workspace, nbytes, dev):
    if workspace is None:
        return alloc_workspace(nbytes, dev)
    if workspace.device != dev:
        raise ValueError(f"workspace: expected a tensor on {dev}, got {workspace.device}")
    # its size is counted in elements: a view that repeats or skips some has other bytes
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace


def _launch(dev, fn, *args):
    """Call fn(*args, stream) with dev's current stream, on dev."""
    import torch
    # the handle of torch.cuda.current_stream(dev), without making a Stream object: 1.8 us
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch._C._cuda_getDevice() == dev.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != FLCE_OK:
        _check(status)


def _mx_format(fmt, allowed=tuple(MX_FORMATS)) -> int:
    if fmt not in allowed:
        raise ValueError(f"microscaled format: expected one of {allowed}, got {fmt!r}")
    return MX_FORMATS[fmt]


def mx_sizes(cols: int, fmt: str) -> Tuple[int, int]:
    """Bytes of a row of codes and of a row of scales for `cols` elements."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(load().flce_mx_sizes(int(cols), _mx_format(fmt), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def _mx_row_bytes(cols, f):
    blocks = -(-cols // 32)
    return blocks * (16 if f == 0 else 32), -(-blocks // 16) * 16


def _mx_empty(rows, cols, fmt, f, dev):
    import torch
    cb, sb = _mx_row_bytes(cols, f)
    # (sizes as plain arguments: torch takes 0.7 us longer over a tuple)
    return MXTensor(torch.empty(rows, cb, dtype=torch.uint8, device=dev),
                    torch.empty(rows, sb, dtype=torch.uint8, device=dev), fmt, cols)


def _mx_check(q, name, dev, f, rows, cols):
    import torch
    cb, sb = _mx_row_bytes(cols, f)
    if q.cols != cols:
        raise ValueError(f"{name}: expected {cols} columns, got {q.cols}")
    for part, t, n in (("codes", q.codes, cb), ("scales", q.scales, sb)):
        if (t.dtype == torch.uint8 and t.device == dev and t.shape == (rows, n)
                and t.is_contiguous()):
            continue
        if t.dtype != torch.uint8:
            raise TypeError(f"{name}.{part}: expected uint8, got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"{name}.{part}: expected a tensor on {dev}, got {t.device}")
        raise ValueError(f"{name}.{part}: expected contiguous shape {(rows, n)}, got "
                         f"{tuple(t.shape)}")


def mx_quantize(x, fmt: str, out: Optional[MXTensor] = None) -> MXTensor:
    """x [rows, cols] (bf16 or fp32) in a microscaled format: "mxfp4", "mxfp8" or "mxint8"."""
    f = _mx_format(fmt)
    if out is None:
        r = _fast().mx_quantize(x, f)
        if r is not None:
            return MXTensor(r[0], r[1], fmt, x.shape[1])
    dev = _on_gpu(x, "x")
    xd, ldx = _dtype_id(x, "x"), _rows(x, "x", dev)
    m, h = x.shape
    if out is None:
        out = _mx_empty(m, h, fmt, f, dev)
    else:
        if out.fmt != fmt:
            raise ValueError(f"out: expected format {fmt}, got {out.fmt}")
        _mx_check(out, "out", dev, f, m, h)
    _launch(dev, load().flce_mx_quantize, x.data_ptr(), xd, ldx, m, h, f, out.codes.data_ptr(),
            out.scales.data_ptr())
    return out


def mx_dequantize(q: MXTensor, dtype=None, out=None):
    """The values of a microscaled matrix, as bf16 (the default) or fp32."""
    f = _mx_format(q.fmt)
    if out is None:
        r = _fast().mx_dequantize(q.codes, q.scales, f, q.cols, dtype)
        if r is not None:
            return r
    import torch
    dev = _on_gpu(q.codes, "codes")
    m = q.codes.shape[0]
    _mx_check(q, "q", dev, f, m, q.cols)
    if out is None:
        out = torch.empty(m, q.cols, dtype=torch.bfloat16 if dtype is None else dtype, device=dev)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out: expected {dtype}, got {out.dtype}")
    od, ldo = _dtype_id(out, "out"), _rows(out, "out", dev, (m, q.cols))
    _launch(dev, load().flce_mx_dequantize, q.codes.data_ptr(), q.scales.data_ptr(), f, m, q.cols,
            out.data_ptr(), od, ldo)
    return out


def _params(weight, bias, dev, h):
    """The parameters' common element type (bf16 without any)."""
    first = bias if weight is None else weight
    if first is None:
        return 0
    pd = _dtype_id(first, "weight" if first is weight else "bias")
    if weight is not None:
        _vector(weight, "weight", dev, first.dtype, h)
    if bias is not None:
        if bias.dtype != first.dtype:
            raise TypeError("weight and bias must have the same dtype")
        _vector(bias, "bias", dev, first.dtype, h)
    return pd


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, out_dtype=None,
                       checkpoint: Optional[str] = None, out=None):
    """(y, mean, rstd) of the layer norm over the rows of x [M, H], and with `checkpoint`
    ("mxfp8" or "mxint8") a fourth result: x in that format, for layer_norm_backward.

    x is bf16 or fp32, y has out_dtype (x's by default; bf16 from fp32 is the usual step from
    an fp32 residual stream into the bf16 head), mean and rstd are fp32 [M].  `out` may supply
    the results' buffers."""
    f = _MX_NONE if checkpoint is None else _mx_format(checkpoint, ("mxfp8", "mxint8"))
    if out is None:
        r = _fast().layer_norm_forward(x, weight, bias, eps, out_dtype, f)
        if r is not None:
            return r if checkpoint is None else (*r[:3], MXTensor(r[3], r[4], checkpoint, x.shape[1]))
    import torch
    dev = _on_gpu(x, "x")
    xd, ldx = _dtype_id(x, "x"), _rows(x, "x", dev)
    m, h = x.shape
    pd = _params(weight, bias, dev, h)
    kept = None
    if out is None:
        if (out_dtype is None or out_dtype == x.dtype) and ldx == h:
            y, yd = torch.empty_like(x), xd
        else:
            y = torch.empty(m, h, dtype=x.dtype if out_dtype is None else out_dtype, device=dev)
            yd = _dtype_id(y, "y")
        ldy = h
        mean = torch.empty(m, dtype=torch.float32, device=dev)
        rstd = torch.empty(m, dtype=torch.float32, device=dev)
        if checkpoint is not None:
            kept = _mx_empty(m, h, checkpoint, f, dev)
    else:
        y, mean, rstd = out[:3]
        if out_dtype is not None and y.dtype != out_dtype:
            raise TypeError(f"y: expected {out_dtype}, got {y.dtype}")
        _vector(mean, "mean", dev, torch.float32, m)
        _vector(rstd, "rstd", dev, torch.float32, m)
        if checkpoint is not None:
            kept = out[3]
            if kept.fmt != checkpoint:
                raise ValueError(f"checkpoint: expected format {checkpoint}, got {kept.fmt}")
            _mx_check(kept, "checkpoint", dev, f, m, h)
        yd, ldy = _dtype_id(y, "y"), _rows(y, "y", dev, (m, h))
    codes, scales = (None, None) if kept is None else (kept.codes.data_ptr(), kept.scales.data_ptr())
    _launch(dev, load().flce_layer_norm_forward, x.data_ptr(), xd, ldx, _ptr(weight), _ptr(bias),
            pd, m, h, eps, y.data_ptr(), yd, ldy, mean.data_ptr(), rstd.data_ptr(), f, codes, scales)
    return (y, mean, rstd) if kept is None else (y, mean, rstd, kept)


@functools.lru_cache(maxsize=256)
def layer_norm_backward_workspace(M: int, H: int) -> int:
    """Workspace bytes of layer_norm_backward."""
    b = ctypes.c_size_t()
    _check(load().flce_layer_norm_backward_workspace(int(M), int(H), ctypes.byref(b)))
    return b.value


def layer_norm_backward(dy, x, mean, rstd, weight=None, dx_dtype=None, need_params: bool = True,
                        param_dtype=None, workspace=None, out=None):
    """(dx, dweight, dbias) of layer_norm_forward; x is its input or its checkpoint.

    dx has x's dtype (from a checkpoint: dx_dtype, dy's by default), dweight and dbias have
    weight's (without one: param_dtype, fp32 by default), or are None without need_params.
    `out` may supply the three buffers."""
    saved = isinstance(x, MXTensor)
    f = _mx_format(x.fmt, ("mxfp8", "mxint8")) if saved else _MX_NONE
    if out is None and workspace is None and (not saved or (dy.dim() == 2 and x.cols == dy.shape[1])):
        r = _fast().layer_norm_backward(
            dy, None if saved else x, x.codes if saved else None, x.scales if saved else None, f,
            mean, rstd, weight, dx_dtype, bool(need_params), param_dtype)
        if r is not None:
            return r
    import torch
    dev = _on_gpu(dy, "dy")
    dyd, lddy = _dtype_id(dy, "dy"), _rows(dy, "dy", dev)
    m, h = dy.shape
    if saved:
        _mx_check(x, "x", dev, f, m, h)
        xp, xd, ldx, codes, scales = None, 0, h, x.codes.data_ptr(), x.scales.data_ptr()
        dx_dtype = dy.dtype if dx_dtype is None else dx_dtype
    else:
        xd, ldx = _dtype_id(x, "x"), _rows(x, "x", dev, (m, h))
        xp, codes, scales = x.data_ptr(), None, None
        if dx_dtype is not None and dx_dtype != x.dtype:
            raise TypeError(f"dx_dtype: expected x's {x.dtype}, got {dx_dtype}")
        dx_dtype = x.dtype
    _vector(mean, "mean", dev, torch.float32, m)
    _vector(rstd, "rstd", dev, torch.float32, m)
    if weight is not None:
        _vector(weight, "weight", dev, weight.dtype, h)
        if param_dtype is not None and param_dtype != weight.dtype:
            raise TypeError(f"param_dtype: expected weight's {weight.dtype}, got {param_dtype}")
        param_dtype = weight.dtype
    elif param_dtype is None:
        param_dtype = torch.float32
    dw = db = None
    if out is None:
        dx = torch.empty(m, h, dtype=dx_dtype, device=dev)
        if need_params:
            dw = torch.empty(h, dtype=param_dtype, device=dev)
            db = torch.empty(h, dtype=param_dtype, device=dev)
    else:
        dx, dw, db = out
        if dx.dtype != dx_dtype:
            raise TypeError(f"dx: expected {dx_dtype}, got {dx.dtype}")
        for name, t in (("dweight", dw), ("dbias", db)):
            if t is not None:
                _vector(t, name, dev, param_dtype, h)
    dxd, lddx = _dtype_id(dx, "dx"), _rows(dx, "dx", dev, (m, h))
    pd = _DTYPE_IDS.get(param_dtype)
    if pd is None:
        raise TypeError(f"param_dtype: expected bfloat16 or float32, got {param_dtype}")
    workspace = _workspace(
        workspace, layer_norm_backward_workspace(m, h) if workspace is None else 0, dev)
    _launch(dev, load().flce_layer_norm_backward, dy.data_ptr(), dyd, lddy, xp, xd, ldx, f, codes,
            scales, _ptr(weight), pd, mean.data_ptr(), rstd.data_ptr(), m, h, dx.data_ptr(), dxd,
            lddx, _ptr(dw), _ptr(db), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dx, dw, db


@functools.lru_cache(maxsize=256)
def mxfp4_workspace_query(M: int, H: int, V: int, compute_entropy: bool = True) -> Tuple[int, int]:
    """Workspace bytes of (mxfp4_logits, mxfp4_forward with every row at once)."""
    lo, fw = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().flce_mx_workspace_query(int(M), int(H), int(V), int(bool(compute_entropy)),
                                          ctypes.byref(lo), ctypes.byref(fw)))
    return lo.value, fw.value


def _plain_head(X, W) -> bool:
    return (isinstance(W, MXTensor) and W.fmt == "mxfp4" and X.dim() == 2
            and W.cols == X.shape[1])


def _mx_head(X, W):
    """Checks shared by the calls of the 4-bit head; returns (device, M, H, V)."""
    import torch
    dev = _on_gpu(X, "X")
    if X.dtype != torch.bfloat16:
        raise TypeError(f"X: expected torch.bfloat16, got {X.dtype}")
    if X.dim() != 2 or not X.is_contiguous():
        raise ValueError("X: expected a contiguous matrix")
    if not isinstance(W, MXTensor) or W.fmt != "mxfp4":
        raise ValueError('W: expected an MXTensor in format "mxfp4" (see mx_quantize)')
    m, h = X.shape
    v = W.codes.shape[0]
    _mx_check(W, "W", dev, 0, v, h)
    return dev, m, h, v


def mxfp4_logits(X, W: MXTensor, scale: float = 1.0, out_dtype=None, workspace=None, out=None):
    """scale * Q(X) W^T [M, V] for a head W in MXFP4, as bf16 (the default) or fp32.

    X [M, H] bf16 is rounded to MXFP4 on the way; sums are in fp32."""
    if out is None and workspace is None and _plain_head(X, W):
        r = _fast().mxfp4_logits(X, W.codes, W.scales, scale, out_dtype)
        if r is not None:
            return r
    import torch
    dev, m, h, v = _mx_head(X, W)
    if out is None:
        out = torch.empty(m, v, dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    od, ldo = _dtype_id(out, "out"), _rows(out, "out", dev, (m, v))
    workspace = _workspace(workspace, mxfp4_workspace_query(m, h, v)[0] if workspace is None else 0, dev)
    _launch(dev, load().flce_mx_logits, X.data_ptr(), W.codes.data_ptr(), W.scales.data_ptr(), m, h,
            v, scale, out.data_ptr(), od, ldo, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return out


def mxfp4_forward(X, W: MXTensor, targets, ignore_index: int = -100, scale: float = 1.0,
                  compute_entropy: bool = True, workspace=None, out=None):
    """forward() with a head in MXFP4: (logprob, lse, entropy-or-None) as fp32 [M] tensors.

    X [M, H] bf16 is rounded to MXFP4 on the way.  Not differentiable."""
    if out is None and workspace is None and _plain_head(X, W):
        r = _fast().mxfp4_forward(X, W.codes, W.scales, targets, ignore_index, scale,
                                  bool(compute_entropy))
        if r is not None:
            return r
    import torch
    dev, m, h, v = _mx_head(X, W)
    _vector(targets, "targets", dev, torch.int64, m)
    if out is None:
        logprob = torch.empty(m, dtype=torch.float32, device=dev)
        lse = torch.empty(m, dtype=torch.float32, device=dev)
        entropy = torch.empty(m, dtype=torch.float32, device=dev) if compute_entropy else None
    else:
        logprob, lse, entropy = out
        for name, t in (("logprob", logprob), ("lse", lse), ("entropy", entropy)):
            if t is not None:
                _vector(t, name, dev, torch.float32, m)
    ent = int(bool(compute_entropy))
    workspace = _workspace(
        workspace, mxfp4_workspace_query(m, h, v, ent)[1] if workspace is None else 0, dev)
    _launch(dev, load().flce_mx_forward, X.data_ptr(), W.codes.data_ptr(), W.scales.data_ptr(),
            targets.data_ptr(), m, h, v, ignore_index, scale, ent, logprob.data_ptr(), lse.data_ptr(),
            _ptr(entropy), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return logprob, lse, entropy


# ----------------------------------------------------------------------------
# the residual block in front of the head: matrix product with an epilogue, dropout
ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation: expected one of {tuple(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _operand(t, name, dev, shape=None):
    """Check a bf16 matrix with contiguous rows; returns its row stride."""
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    return _rows(t, name, dev, shape)


def _result(out, name, dtype, dev, shape, what):
    """A result's buffer: a new one, or the caller's, checked; with its type's id and row stride."""
    import torch
    if out is None:
        out = torch.empty(*shape, dtype=dtype, device=dev)
    elif out.dtype != dtype:
        raise TypeError(f"{name}: expected {what} {dtype}, got {out.dtype}")
    return out, _dtype_id(out, name), _rows(out, name, dev, shape)


@functools.lru_cache(maxsize=256)
def linear_workspace(M: int, N: int, K: int) -> Tuple[int, int]:
    """Workspace bytes of (linear_forward, linear_backward)."""
    fw, bw = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().flce_linear_workspace(int(M), int(N), int(K), ctypes.byref(fw), ctypes.byref(bw)))
    return fw.value, bw.value


def linear_forward(X, W, bias=None, activation: Optional[str] = None, residual=None, out_dtype=None,
                   keep_pre: bool = False, workspace=None, out=None):
    """act(X W^T + bias) + residual [M, N], bf16 (the default) or fp32; with keep_pre the pair of it
    and X W^T + bias in bf16, for linear_backward.

    X [M, K] and W [N, K] are bf16 with 16-byte aligned rows, bias [N] and residual [M, N] bf16 or
    fp32; activation is None, "relu", "gelu", "gelu_tanh" or "silu".  `out` may supply the result's
    buffer (with keep_pre the pair), and may be residual."""
    act = _activation(activation)
    if out is None and workspace is None:
        r = _fast().linear_forward(X, W, bias, act, residual, out_dtype, bool(keep_pre))
        if r is not None:
            return r
    import torch
    dev = _on_gpu(X, "X")
    ldx = _operand(X, "X", dev)
    m, k = X.shape
    ldw = _operand(W, "W", dev)
    n = W.shape[0]
    if W.shape[1] != k:
        raise ValueError(f"W: expected {k} columns, got {W.shape[1]}")
    bd = rd = 0
    ldr = n
    if bias is not None:
        bd = _dtype_id(bias, "bias")
        _vector(bias, "bias", dev, bias.dtype, n)
    if residual is not None:
        rd, ldr = _dtype_id(residual, "residual"), _rows(residual, "residual", dev, (m, n))
    out, pre = out if keep_pre and out is not None else (out, None)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    out, od, ldo = _result(out, "out", out_dtype, dev, (m, n), "out_dtype")
    ldp = n
    if keep_pre:
        pre, _, ldp = _result(pre, "pre", torch.bfloat16, dev, (m, n), "")
    workspace = _workspace(workspace, linear_workspace(m, n, k)[0] if workspace is None else 0, dev)
    _launch(dev, load().flce_linear_forward, X.data_ptr(), ldx, W.data_ptr(), ldw, _ptr(bias), bd, act,
            _ptr(residual), rd, ldr, m, n, k, out.data_ptr(), od, ldo, _ptr(pre), ldp,
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return (out, pre) if keep_pre else out


def linear_backward(dy, X, W, pre=None, activation: Optional[str] = None, need_dx: bool = True,
                    need_dw: bool = True, bias_dtype=None, workspace=None, out=None):
    """(dX, dW, dbias) of linear_forward, from dy [M, N] (bf16 or fp32) and, with an activation,
    the forward's pre.  dX and dW are bf16, or None where they are not needed; dbias has bias_dtype
    (None: no dbias).  The gradient of the residual is dy.  `out` may supply the three buffers."""
    act = _activation(activation)
    if out is None and workspace is None:
        r = _fast().linear_backward(dy, X, W, pre, act, bool(need_dx), bool(need_dw), bias_dtype)
        if r is not None:
            return r
    import torch
    dev = _on_gpu(dy, "dy")
    dyd, lddy = _dtype_id(dy, "dy"), _rows(dy, "dy", dev)
    m, n = dy.shape
    ldx, ldw = _operand(X, "X", dev), _operand(W, "W", dev)
    k = X.shape[1]
    if X.shape[0] != m:
        raise ValueError(f"X: expected {m} rows, got {X.shape[0]}")
    if W.shape != (n, k):
        raise ValueError(f"W: expected shape {(n, k)}, got {tuple(W.shape)}")
    ldp = n
    if act:
        if pre is None:
            raise ValueError("pre: needed with an activation (see keep_pre of linear_forward)")
        ldp = _operand(pre, "pre", dev, (m, n))
    dx, dw, db = (None, None, None) if out is None else out
    lddx = lddw = k
    if need_dx:
        dx, _, lddx = _result(dx, "dX", torch.bfloat16, dev, (m, k), "")
    if need_dw:
        dw, _, lddw = _result(dw, "dW", torch.bfloat16, dev, (n, k), "")
    bd = 0
    if bias_dtype is not None:
        if db is None:
            db = torch.empty(n, dtype=bias_dtype, device=dev)
        bd = _dtype_id(db, "dbias")
        _vector(db, "dbias", dev, bias_dtype, n)
    else:
        db = None
    workspace = _workspace(workspace, linear_workspace(m, n, k)[1] if workspace is None else 0, dev)
    _launch(dev, load().flce_linear_backward, dy.data_ptr(), dyd, lddy, _ptr(pre) if act else None, ldp,
            act, X.data_ptr(), ldx, W.data_ptr(), ldw, m, n, k, _ptr(dx) if need_dx else None, lddx,
            _ptr(dw) if need_dw else None, lddw, _ptr(db), bd, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return dx if need_dx else None, dw if need_dw else None, db


def _uint64(v, name) -> int:
    v = int(v)
    if not 0 <= v < 1 << 64:
        raise ValueError(f"{name}: expected 0 <= {name} < 2^64, got {v}")
    return v


def dropout(x, p: float, seed, offset: int = 0, residual=None, out_dtype=None, out=None):
    """residual + dropout(x) over a matrix [M, H]: an element is dropped with probability p (in steps
    of 1 / 65536), and what is kept divided by the probability of that.

    The mask follows from seed, offset and the element's place (include/flce.h), so it is not
    kept: dropout_backward forms it again.  seed is an int, or an int64 GPU tensor of one element
    that the kernel reads (so that a captured call draws anew where its caller writes there);
    offset tells calls with one seed apart.  x and residual are bf16 or fp32; the result has
    out_dtype, by default residual's dtype or x's.  `out` may supply its buffer, and may be x or
    residual."""
    if out is None:
        r = _fast().dropout(x, p, seed, offset, residual, out_dtype)
        if r is not None:
            return r
    import torch
    dev = _on_gpu(x, "x")
    xd, ldx = _dtype_id(x, "x"), _rows(x, "x", dev)
    m, h = x.shape
    rd, ldr = 0, h
    if residual is not None:
        rd, ldr = _dtype_id(residual, "residual"), _rows(residual, "residual", dev, (m, h))
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else x.dtype if residual is None else residual.dtype
    out, yd, ldy = _result(out, "out", out_dtype, dev, (m, h), "out_dtype")
    at = None
    if isinstance(seed, torch.Tensor):
        _vector(seed.reshape(-1), "seed", dev, torch.int64, 1)
        seed, at = 0, seed.data_ptr()
    _launch(dev, load().flce_dropout, x.data_ptr(), xd, ldx, _ptr(residual), rd, ldr, m, h, float(p),
            _uint64(seed, "seed"), at, _uint64(offset, "offset"), out.data_ptr(), yd, ldy)
    return out


def dropout_backward(dy, p: float, seed, offset: int = 0, dx_dtype=None, out=None):
    """Gradient of dropout's x (dx_dtype: dy's by default) with the forward's p, seed and offset.
    The gradient of residual is dy."""
    return dropout(dy, p, seed, offset, None, dx_dtype, out)


# ----------------------------------------------------------------------------
# log-probs, entropy and alternatives from logits
class TokenLogprobs(NamedTuple):
    """Results of token_logprobs: per given token, per row, and per alternative."""
    logprob: Any
    lse: Any
    entropy: Any
    top_ids: Any
    top_logprob: Any
    stats: Any


@functools.lru_cache(maxsize=256)
def token_logprobs_workspace(M: int, V: int, n_top: int = 0) -> int:
    """Workspace bytes of token_logprobs."""
    b = ctypes.c_size_t()
    _check(load().flce_token_logprobs_workspace(int(M), int(V), int(n_top), ctypes.byref(b)))
    return b.value


def _tokens(tokens, dev, m):
    """Check given tokens [M] or [M, n]; returns their shape and n."""
    import torch
    if tokens is None:
        return (m, 0), 0
    if tokens.dtype != torch.int64:
        raise TypeError(f"tokens: expected torch.int64, got {tokens.dtype}")
    if tokens.device != dev:
        raise ValueError(f"tokens: expected a tensor on {dev}, got {tokens.device}")
    shape = tuple(tokens.shape)
    if len(shape) not in (1, 2) or shape[0] != m or not tokens.is_contiguous():
        raise ValueError(f"tokens: expected {m} contiguous rows, got shape {shape}")
    return shape, 1 if len(shape) == 1 else shape[1]


def _contiguous(t, name, dev, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name}: expected a tensor on {dev}, got {t.device}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def token_logprobs(logits, tokens=None, ignore_index: int = -100, scale: float = 1.0, n_top: int = 0,
                   compute_entropy: bool = True, workspace=None, out: Optional[TokenLogprobs] = None):
    """Log-probs of given tokens, log-sum-exp, entropy and the n_top largest alternatives of each row
    of logits [M, V] (bf16 or fp32) under softmax(scale * logits), as a TokenLogprobs.

    tokens are int64 [M] or [M, n]; logprob has their shape (0 where a token is ignore_index or
    outside [0, V); [M, 0] without tokens).  top_ids int64 and top_logprob [M, n_top] are ordered by
    the logits, equal ones by index; a logit of -inf is masked.  entropy is None without
    compute_entropy, the alternatives without n_top.  stats [M, 2] is what
    token_logprobs_backward needs of the rows.  `out` may supply the buffers."""
    if out is None and workspace is None:
        r = _fast().token_logprobs(logits, tokens, ignore_index, scale, n_top, bool(compute_entropy))
        if r is not None:
            return TokenLogprobs(*r)
    import torch
    dev = _on_gpu(logits, "logits")
    d, ldl = _dtype_id(logits, "logits"), _rows(logits, "logits", dev)
    m, v = logits.shape
    shape, n = _tokens(tokens, dev, m)
    n_top = int(n_top)
    f32, f = torch.float32, functools.partial(torch.empty, device=dev)
    if out is None:
        out = TokenLogprobs(f(shape, dtype=f32), f(m, dtype=f32), f(m, dtype=f32) if compute_entropy else None,
                            f(m, n_top, dtype=torch.int64) if n_top > 0 else None,
                            f(m, n_top, dtype=f32) if n_top > 0 else None, f(m, 2, dtype=f32))
    else:
        _contiguous(out.logprob, "logprob", dev, f32, shape)
        _contiguous(out.lse, "lse", dev, f32, (m,))
        _contiguous(out.stats, "stats", dev, f32, (m, 2))
        if compute_entropy:
            _contiguous(out.entropy, "entropy", dev, f32, (m,))
        if n_top > 0:
            _contiguous(out.top_ids, "top_ids", dev, torch.int64, (m, n_top))
            _contiguous(out.top_logprob, "top_logprob", dev, f32, (m, n_top))
    workspace = _workspace(
        workspace, token_logprobs_workspace(m, v, n_top) if workspace is None and v else 0, dev)
    _launch(dev, load().flce_token_logprobs, logits.data_ptr(), d, ldl, m, v, _ptr(tokens), n, ignore_index,
            scale, n_top, out.logprob.data_ptr(), out.lse.data_ptr(),
            _ptr(out.entropy) if compute_entropy else None, out.stats.data_ptr(), _ptr(out.top_ids),
            _ptr(out.top_logprob), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def token_logprobs_backward(logits, tokens, stats, entropy=None, top_ids=None, grad_logprob=None,
                            grad_top=None, grad_entropy=None, grad_lse=None,
                            ignore_index: int = -100, scale: float = 1.0, out=None):
    """dlogits (logits' dtype) of token_logprobs, from the gradients of logprob, of top_logprob (with
    the forward's top_ids), of entropy (with the forward's entropy) and of lse; None counts as 0.  `out` may
    supply its buffer, and may be logits."""
    if out is None:
        r = _fast().token_logprobs_backward(logits, tokens, stats, entropy, top_ids, grad_logprob, grad_top,
                                            grad_entropy, grad_lse, ignore_index, scale)
        if r is not None:
            return r
    import torch
    dev = _on_gpu(logits, "logits")
    d, ldl = _dtype_id(logits, "logits"), _rows(logits, "logits", dev)
    m, v = logits.shape
    shape, n = _tokens(tokens, dev, m)
    f32 = torch.float32
    _contiguous(stats, "stats", dev, f32, (m, 2))
    if grad_logprob is not None:
        _contiguous(grad_logprob, "grad_logprob", dev, f32, shape)
    n_top = 0
    if grad_top is not None:
        if top_ids is None:
            raise ValueError("top_ids: needed with grad_top")
        if top_ids.dim() != 2:
            raise ValueError(f"top_ids: expected a matrix, got {top_ids.dim()} dimensions")
        n_top = top_ids.shape[1]
        _contiguous(top_ids, "top_ids", dev, torch.int64, (m, n_top))
        _contiguous(grad_top, "grad_top", dev, f32, (m, n_top))
    if grad_entropy is not None:
        if entropy is None:
            raise ValueError("entropy: needed with grad_entropy")
        _vector(entropy, "entropy", dev, f32, m)
        _vector(grad_entropy, "grad_entropy", dev, f32, m)
    if grad_lse is not None:
        _vector(grad_lse, "grad_lse", dev, f32, m)
    out, _, ldd = _result(out, "out", logits.dtype, dev, (m, v), "logits'")
    _launch(dev, load().flce_token_logprobs_backward, logits.data_ptr(), d, ldl, m, v, _ptr(tokens), n,
            ignore_index, scale, stats.data_ptr(), _ptr(entropy) if grad_entropy is not None else None,
            _ptr(top_ids) if n_top else None, n_top, _ptr(grad_logprob), _ptr(grad_top) if n_top else None,
            _ptr(grad_entropy), _ptr(grad_lse), out.data_ptr(), ldd)
    return out
