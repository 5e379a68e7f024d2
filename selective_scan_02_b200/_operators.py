"""Binding of libss2d.so's operators of a linear-attention layer: argument marshalling only.

As in _binding.py, every function checks its tensors, passes pointers, sizes and a stream to
the C ABI of include/ss2d.h and computes nothing itself; here a compiled module does so
(csrc/marshal.cpp), because these calls are short.  All tensors of a call are on one CUDA
device, which need not be the current one; the work is enqueued on `stream`, or on that
device's current stream.  Outputs and workspaces allocated here belong to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import Ss2dError, _check, load_library

SS2D_E4M3 = 2


class MatmulFp8Args(ctypes.Structure):
    """Mirror of ss2d_matmul_fp8_args (include/ss2d.h)."""

    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
        ("a", ctypes.c_void_p), ("a_scales", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("w_scales", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("c", ctypes.c_void_p), ("c_dtype", ctypes.c_int),
    ]


class LinearAttentionArgs(ctypes.Structure):
    """Mirror of ss2d_linear_attention_args (include/ss2d.h)."""

    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", ctypes.c_int), ("L", ctypes.c_int), ("G", ctypes.c_int), ("H", ctypes.c_int),
        ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3), ("v_stride", ctypes.c_longlong * 3),
        ("log_decay", ctypes.c_void_p), ("decay_per_token", ctypes.c_int),
        ("lengths", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("h0", ctypes.c_void_p), ("h_last", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
    ]


class LinearAttentionStepArgs(ctypes.Structure):
    """Mirror of ss2d_linear_attention_step_args (include/ss2d.h)."""

    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", ctypes.c_int), ("pool", ctypes.c_int), ("G", ctypes.c_int), ("H", ctypes.c_int),
        ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong * 2), ("k_stride", ctypes.c_longlong * 2), ("v_stride", ctypes.c_longlong * 2),
        ("log_decay", ctypes.c_void_p), ("decay_per_token", ctypes.c_int),
        ("slots", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("state", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
    ]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.ss2d_rms_norm.argtypes = [P, I, P, I, P, ctypes.c_float, P, I, P, P, ctypes.c_longlong, I, P]
        lib.ss2d_rms_norm.restype = I
        lib.ss2d_matmul_fp8_workspace.argtypes = [ctypes.POINTER(MatmulFp8Args)]
        lib.ss2d_matmul_fp8_workspace.restype = S
        lib.ss2d_matmul_fp8.argtypes = [ctypes.POINTER(MatmulFp8Args), P, S, P]
        lib.ss2d_matmul_fp8.restype = I
        lib.ss2d_linear_attention_workspace.argtypes = [ctypes.POINTER(LinearAttentionArgs)]
        lib.ss2d_linear_attention_workspace.restype = S
        lib.ss2d_linear_attention.argtypes = [ctypes.POINTER(LinearAttentionArgs), P, S, P]
        lib.ss2d_linear_attention.restype = I
        lib.ss2d_linear_attention_step.argtypes = [ctypes.POINTER(LinearAttentionStepArgs), P]
        lib.ss2d_linear_attention_step.restype = I
        lib.ss2d_workspace_status.argtypes = [P, P]
        lib.ss2d_workspace_status.restype = I
        lib.ss2d_wait_status.argtypes = [P]
        lib.ss2d_wait_status.restype = I
        lib.ss2d_diag_operator_wait.argtypes = [P, ctypes.c_longlong, P]
        lib.ss2d_diag_operator_wait.restype = I
        _lib = lib
    return _lib


_marshal = None


def _module():
    """The compiled marshalling module (csrc/marshal.cpp), which calls libss2d.so."""
    global _marshal
    if _marshal is None:
        load_library()  # says so if libss2d.so is missing
        from . import _marshal as module

        _marshal = module
    return _marshal


def _size(n):
    if n == ctypes.c_size_t(-1).value:
        raise Ss2dError(1, "SS2D_ERR_INVALID_ARG", _library().ss2d_last_error().decode())
    return int(n)


def _on_stream(stream, call, x, *rest):
    """call(x, *rest) on `stream`: what it allocates belongs to that stream, and is kept from reuse until
    the work that the current stream holds at its release is done."""
    if not isinstance(x, torch.Tensor) or stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are not")
    current = torch.cuda.current_stream(x.device)
    if stream.cuda_stream == current.cuda_stream:
        return call(x, *rest)
    with torch.cuda.stream(stream):
        got = call(x, *rest)
    given = {id(t) for t in (x, *rest)}
    for t in got if isinstance(got, tuple) else (got,):
        if isinstance(t, torch.Tensor) and id(t) not in given:
            t.record_stream(current)
    return got


def rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=torch.bfloat16, y=None, scales=None, residual_out=None,
             stream=None):
    """Root-mean-square norm with the residual's addition (ss2d_rms_norm).

    x (..., D) fp32 or bf16, weight (D) fp32, residual (..., D) fp32 or bf16 or None:
    r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight in fp32.  Returns y, or a tuple
    of y, then scales if y is float8_e4m3fn, then residual_out (r in the residual's type) if a
    residual is given.  out_dtype (float32, bfloat16 or float8_e4m3fn) is the type of a y
    allocated here; a given y keeps its own.  scales (..., ceil(D / 128)) fp32 holds one scale
    for each 128 columns of a row.  residual_out may be `residual` itself.  A row's sum of r^2 must
    be below 2^128.
    """
    call = (_marshal or _module()).rms_norm
    if stream is None:
        got = call(x, weight, residual, eps, out_dtype, y, scales, residual_out)
    else:
        got = _on_stream(stream, call, x, weight, residual, eps, out_dtype, y, scales, residual_out)
    return got if got.__class__ is not int else _check(got, "ss2d_rms_norm")


def matmul_fp8(a, a_scales, w, w_scales, bias=None, out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """Product of e4m3 matrices with a scale for each block of 128 (ss2d_matmul_fp8):
    (..., N) = (a * a_scales) (w * w_scales)^T + bias.

    a (..., K) float8_e4m3fn with a_scales (..., ceil(K / 128)) fp32, as rms_norm returns them;
    w (N, K) float8_e4m3fn with w_scales (ceil(N / 128), ceil(K / 128)) fp32; bias (N) fp32
    or None.  K is a multiple of 16.  out_dtype (bfloat16 or float32) is the type of an out
    allocated here; a given out keeps its own.  workspace: a tensor of at least
    matmul_fp8_workspace_size bytes, not shared by calls that overlap on the GPU; allocated here
    when none is given.
    """
    call = (_marshal or _module()).matmul_fp8
    if stream is None:
        got = call(a, a_scales, w, w_scales, bias, out_dtype, out, workspace)
    else:
        got = _on_stream(stream, call, a, a_scales, w, w_scales, bias, out_dtype, out, workspace)
    return got if got.__class__ is not int else _check(got, "ss2d_matmul_fp8")


def matmul_fp8_workspace_size(M, N, K) -> int:
    """Workspace bytes ss2d_matmul_fp8 needs for these sizes."""
    n = _library().ss2d_matmul_fp8_workspace(MatmulFp8Args(ctypes.sizeof(MatmulFp8Args), M, N, K))
    return _size(n)


def linear_attention(q, k, v, log_decay, scale=1.0, h0=None, lengths=None, return_last_state=False, out=None,
                     h_last=None, workspace=None, stream=None):
    """Causal linear attention with a decay for each head over whole sequences (ss2d_linear_attention).

    For each sequence and head, S <- exp(log_decay) S + k_t v_t^T and o_t = scale * S^T q_t.
    q, k (B, L, G, Dk) and v (B, L, H, Dv) bf16, with any strides that keep 16-byte rows (columns
    of one projection's output, for instance); H is a multiple of G, Dk and Dv multiples of 8 up
    to 128.  log_decay (H) or (B, L, H) fp32, at most 0.  h0 (B, H, Dk, Dv) fp32 is the state
    before the first token (None: zero).  lengths (B) int32: the tokens of each sequence; rows of
    `out` behind them are left as they were.  Returns out (B, L, H, Dv) bf16, or (out, h_last)
    with return_last_state or an h_last given (which may be h0 itself).  workspace: a tensor of
    at least linear_attention_workspace_size bytes, not shared by calls that overlap on the GPU;
    allocated here when none is given.  States and sums are fp32; above 8 tokens, scores and the
    state enter `out` rounded to bf16.
    """
    call = (_marshal or _module()).linear_attention
    if stream is None:
        got = call(q, k, v, log_decay, scale, h0, lengths, return_last_state, out, h_last, workspace)
    else:
        got = _on_stream(stream, call, q, k, v, log_decay, scale, h0, lengths, return_last_state, out, h_last, workspace)
    return got if got.__class__ is not int else _check(got, "ss2d_linear_attention")


def linear_attention_workspace_size(B, L, G, H, Dk, Dv) -> int:
    """Workspace bytes ss2d_linear_attention needs for these sizes."""
    args = LinearAttentionArgs(ctypes.sizeof(LinearAttentionArgs), B, L, G, H, Dk, Dv)
    return _size(_library().ss2d_linear_attention_workspace(args))


def linear_attention_step(q, k, v, log_decay, state, slots=None, scale=1.0, out=None, stream=None):
    """One new token of each of B rows (ss2d_linear_attention_step): state is updated in place and
    out (B, H, Dv) bf16 returned.

    q, k (B, G, Dk) and v (B, H, Dv) bf16 (strided as for linear_attention); log_decay (H) or
    (B, H) fp32; state (pool, H, Dk, Dv) fp32.  slots (B) int32 names the state of each row
    (None: row b has state b); a row whose slot is outside the pool is empty and its row of `out`
    is left as it was, and rows of one slot are consecutive tokens in the order of the rows (at
    most 65536 rows with slots).
    """
    call = (_marshal or _module()).linear_attention_step
    if stream is None:
        got = call(q, k, v, log_decay, state, slots, scale, out)
    else:
        got = _on_stream(stream, call, q, k, v, log_decay, state, slots, scale, out)
    return got if got.__class__ is not int else _check(got, "ss2d_linear_attention_step")


def check_workspace_status(workspace=None, stream=None):
    """Raises Ss2dError (SS2D_ERR_DEVICE) if a tensor-core kernel's bounded wait ran out: in the last
    matmul_fp8 or linear_attention on `workspace` (ss2d_workspace_status), or, with none, in any such call on the
    stream's device (the current one), with workspaces of whatever origin, since this was last reported
    (ss2d_wait_status).  Synchronises the stream."""
    if workspace is None:
        stream = torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.device(stream.device):
            _check(_library().ss2d_wait_status(ctypes.c_void_p(stream.cuda_stream)), "ss2d_wait_status")
        return
    got = _module().workspace_status(workspace) if stream is None else _on_stream(
        stream, _module().workspace_status, workspace)
    _check(got, "ss2d_workspace_status")


def diag_operator_wait(workspace, spin_limit, stream=None):
    """ss2d_diag_operator_wait: the operators' tensor-core waits run out on purpose after spin_limit polls, which is
    noted in the workspace's error word and the device's (for testing failure reporting)."""
    if not workspace.is_cuda or not workspace.is_contiguous() or workspace.nbytes < 4:
        raise ValueError("workspace must be a contiguous device tensor of at least 4 bytes")
    with torch.cuda.device(workspace.device):
        stream = torch.cuda.current_stream() if stream is None else stream
        _check(_library().ss2d_diag_operator_wait(workspace.data_ptr(), int(spin_limit), ctypes.c_void_p(stream.cuda_stream)),
               "ss2d_diag_operator_wait")
