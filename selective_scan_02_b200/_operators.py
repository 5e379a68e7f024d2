"""ctypes binding of libss2d.so's operators of a linear-attention layer: argument marshalling only.

As in _binding.py, every function checks its tensors, passes pointers, sizes and a stream to
the C ABI of include/ss2d.h and computes nothing itself.  All tensors of a call are on one CUDA
device, which need not be the current one; the work is enqueued on `stream`, or on that
device's current stream.  Outputs and workspaces allocated here belong to that stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import SS2D_BF16, SS2D_F32, Ss2dError, _check, load_library

SS2D_E4M3 = 2
FP8_BLOCK = 128
_NO_SIZE = ctypes.c_size_t(-1).value
_OUT_CODE = {torch.float32: SS2D_F32, torch.bfloat16: SS2D_BF16, torch.float8_e4m3fn: SS2D_E4M3}


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


_MATMUL_SIZE = ctypes.sizeof(MatmulFp8Args)
_ATTENTION_SIZE = ctypes.sizeof(LinearAttentionArgs)
_STEP_SIZE = ctypes.sizeof(LinearAttentionStepArgs)
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
        _lib = lib
    return _lib


class _Call:
    """The device and stream of one call: `with _Call(x, stream) as c` makes the device current
    and c.new(...) allocates on the call's stream."""

    __slots__ = ("index", "device", "handle", "_stream", "_guard")

    def __init__(self, t, stream):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError("libss2d takes device tensors")
        self.device = t.device
        self.index = t.get_device()
        self.handle = torch._C._cuda_getCurrentRawStream(self.index)
        self._stream = self._guard = None
        if stream is not None:
            if stream.device != self.device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {self.device}")
            if stream.cuda_stream != self.handle:
                self.handle = stream.cuda_stream
                self._stream = stream

    def __enter__(self):
        if self.index != torch._C._cuda_getDevice():
            self._guard = torch.cuda.device(self.index)
            self._guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)

    def new(self, shape, dtype):
        if self._stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self._stream):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.index))
        return t

    def like(self, t, dtype):
        """new(t.shape, dtype) of a dense t."""
        return torch.empty_like(t, dtype=dtype) if self._stream is None else self.new(t.shape, dtype)

    def ptr(self, t, name, dtype, shape):
        """The pointer of a dense tensor of this device, type and shape; None stays None."""
        if t is None:
            return None
        if t.get_device() != self.index or t.dtype != dtype or t.shape != shape:
            self._refuse(t, name, dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def strided(self, t, name, shape):
        """Pointer and strides of a bf16 tensor with a dense last dimension."""
        if t.get_device() != self.index or t.dtype != torch.bfloat16 or t.shape != shape:
            self._refuse(t, name, torch.bfloat16, shape)
        strides = t.stride()
        if strides[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"the last dimension of {name} must be dense")
        return t.data_ptr(), strides

    def _refuse(self, t, name, dtype, shape):
        if t.get_device() != self.index:
            raise ValueError(f"{name} is on {t.device}, not on {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {str(dtype).removeprefix('torch.')}")
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _float_code(t, name):
    code = _OUT_CODE.get(t.dtype)
    if code is None or code == SS2D_E4M3:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code


def _workspace(call, workspace, need):
    if not need:
        return None, 0, None  # the call itself says what is wrong with its arguments
    if workspace is None:
        workspace = call.new((need,), torch.uint8)
        return workspace.data_ptr(), need, workspace
    if workspace.get_device() != call.index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {call.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=torch.bfloat16, y=None, scales=None, residual_out=None,
             stream=None):
    """Root-mean-square norm with the residual's addition (ss2d_rms_norm).

    x (..., D) fp32 or bf16, weight (D) fp32, residual (..., D) fp32 or bf16 or None:
    r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight in fp32.  Returns y, or a tuple
    of y, then scales if y is float8_e4m3fn, then residual_out (r in the residual's type) if a
    residual is given.  out_dtype (float32, bfloat16 or float8_e4m3fn) is the type of a y
    allocated here; a given y keeps its own.  scales (..., ceil(D / 128)) fp32 holds one scale
    for each 128 columns of a row.  residual_out may be `residual` itself.
    """
    with _Call(x, stream) as c:
        shape = x.shape
        if not shape:
            raise ValueError("x must have a last dimension")
        D = shape[-1]
        rows = x.numel() // D if D else 0
        xc = _float_code(x, "x")
        xp = c.ptr(x, "x", x.dtype, shape)
        wp = c.ptr(weight, "weight", torch.float32, (D,))
        rp, rc, rop = None, 0, None
        if residual is not None:
            rc = _float_code(residual, "residual")
            rp = c.ptr(residual, "residual", residual.dtype, shape)
            if residual_out is None:
                residual_out = c.like(residual, residual.dtype)
                rop = residual_out.data_ptr()
            else:
                rop = c.ptr(residual_out, "residual_out", residual.dtype, shape)
        elif residual_out is not None:
            raise ValueError("residual_out is given without a residual")
        if y is None:
            code = _OUT_CODE.get(out_dtype)
            if code is None:
                raise ValueError("out_dtype must be float32, bfloat16 or float8_e4m3fn")
            y = c.like(x, out_dtype)
            yp = y.data_ptr()
        else:
            code = _OUT_CODE.get(y.dtype)
            if code is None:
                raise ValueError("y must be float32, bfloat16 or float8_e4m3fn")
            yp = c.ptr(y, "y", y.dtype, shape)
        sp = None
        if code == SS2D_E4M3:
            groups = shape[:-1] + (-(-D // FP8_BLOCK),)
            if scales is None:
                scales = c.new(groups, torch.float32)
            sp = c.ptr(scales, "scales", torch.float32, groups)
        elif scales is not None:
            raise ValueError("scales is given without a float8_e4m3fn y")
        status = _library().ss2d_rms_norm(xp, xc, rp, rc, wp, eps, yp, code, sp, rop, rows, D, c.handle)
        if status:
            _check(status, "ss2d_rms_norm")
    if residual is None:
        return y if scales is None else (y, scales)
    return (y, residual_out) if scales is None else (y, scales, residual_out)


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
    with _Call(a, stream) as c:
        if a.dim() < 1 or w.dim() != 2:
            raise ValueError("a must be (..., K) and w (N, K)")
        lead, K, N = a.shape[:-1], a.shape[-1], w.shape[0]
        M = a.numel() // K if K else 0
        if max(M, N, K) > 0x7fffffff:
            raise ValueError("sizes must fit 32 bits")
        if out is not None:
            out_dtype = out.dtype
        code = _OUT_CODE.get(out_dtype)
        if code is None or code == SS2D_E4M3:
            raise ValueError("out must be float32 or bfloat16")
        kb, nb = -(-K // FP8_BLOCK), -(-N // FP8_BLOCK)
        ap = c.ptr(a, "a", torch.float8_e4m3fn, a.shape)
        asp = c.ptr(a_scales, "a_scales", torch.float32, lead + (kb,))
        wp = c.ptr(w, "w", torch.float8_e4m3fn, (N, K))
        wsp = c.ptr(w_scales, "w_scales", torch.float32, (nb, kb))
        bp = c.ptr(bias, "bias", torch.float32, (N,))
        if out is None:
            out = c.new(lead + (N,), out_dtype)
        op = c.ptr(out, "out", out_dtype, lead + (N,))
        args = MatmulFp8Args(_MATMUL_SIZE, M, N, K, ap, asp, wp, wsp, bp, op, code)
        lib = _library()
        sp, sn, workspace = _workspace(c, workspace, _matmul_need(M, N, K))
        status = lib.ss2d_matmul_fp8(args, sp, sn, c.handle)
        if status:
            _check(status, "ss2d_matmul_fp8")
    return out


@functools.lru_cache(maxsize=4096)
def _matmul_need(M, N, K):
    """Workspace bytes for these sizes, or 0 if they are refused."""
    n = _library().ss2d_matmul_fp8_workspace(MatmulFp8Args(_MATMUL_SIZE, M, N, K))
    return 0 if n == _NO_SIZE else n


def matmul_fp8_workspace_size(M, N, K) -> int:
    """Workspace bytes ss2d_matmul_fp8 needs for these sizes."""
    n = _matmul_need(M, N, K)
    if not n:
        raise Ss2dError(1, "SS2D_ERR_INVALID_ARG", f"sizes M={M} N={N} K={K} are refused")
    return n


def _heads(q, k, v, lead):
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        names = "(B, L, G, Dk) and (B, L, H, Dv)" if lead == 2 else "(B, G, Dk) and (B, H, Dv)"
        raise ValueError(f"q, k and v must be {names}")
    return q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1]


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
    allocated here when none is given.
    """
    with _Call(q, stream) as c:
        G, H, Dk, Dv = _heads(q, k, v, 2)
        B, L = q.shape[:2]
        qp, qs = c.strided(q, "q", (B, L, G, Dk))
        kp, ks = c.strided(k, "k", (B, L, G, Dk))
        vp, vs = c.strided(v, "v", (B, L, H, Dv))
        per_token = log_decay.dim() == 3
        gp = c.ptr(log_decay, "log_decay", torch.float32, (B, L, H) if per_token else (H,))
        lp = c.ptr(lengths, "lengths", torch.int32, (B,))
        state = (B, H, Dk, Dv)
        hp = c.ptr(h0, "h0", torch.float32, state)
        if h_last is None and return_last_state:
            h_last = c.new(state, torch.float32)
        hlp = c.ptr(h_last, "h_last", torch.float32, state)
        if out is None:
            out = c.new((B, L, H, Dv), torch.bfloat16)
        op = c.ptr(out, "out", torch.bfloat16, (B, L, H, Dv))
        a = LinearAttentionArgs(_ATTENTION_SIZE, B, L, G, H, Dk, Dv, qp, kp, vp, qs[:3], ks[:3], vs[:3], gp,
                                per_token, lp, scale, hp, hlp, op)
        lib = _library()
        wp, wn, workspace = _workspace(c, workspace, _attention_need(B, L, G, H, Dk, Dv))
        status = lib.ss2d_linear_attention(a, wp, wn, c.handle)
        if status:
            _check(status, "ss2d_linear_attention")
    return out if h_last is None else (out, h_last)


@functools.lru_cache(maxsize=4096)
def _attention_need(*sizes):
    n = _library().ss2d_linear_attention_workspace(LinearAttentionArgs(_ATTENTION_SIZE, *sizes))
    return 0 if n == _NO_SIZE else n


def linear_attention_workspace_size(B, L, G, H, Dk, Dv) -> int:
    """Workspace bytes ss2d_linear_attention needs for these sizes."""
    n = _attention_need(B, L, G, H, Dk, Dv)
    if not n:
        raise Ss2dError(1, "SS2D_ERR_INVALID_ARG", f"sizes B={B} L={L} G={G} H={H} Dk={Dk} Dv={Dv} are refused")
    return n


def linear_attention_step(q, k, v, log_decay, state, slots=None, scale=1.0, out=None, stream=None):
    """One new token of each of B rows (ss2d_linear_attention_step): state is updated in place and
    out (B, H, Dv) bf16 returned.

    q, k (B, G, Dk) and v (B, H, Dv) bf16 (strided as for linear_attention); log_decay (H) or
    (B, H) fp32; state (pool, H, Dk, Dv) fp32.  slots (B) int32 names the state of each row
    (None: row b has state b); a row whose slot is outside the pool is empty and its row of `out`
    is left as it was, and rows of one slot are consecutive tokens in the order of the rows.
    """
    with _Call(q, stream) as c:
        G, H, Dk, Dv = _heads(q, k, v, 1)
        B, pool = q.shape[0], state.shape[0]
        qp, qs = c.strided(q, "q", (B, G, Dk))
        kp, ks = c.strided(k, "k", (B, G, Dk))
        vp, vs = c.strided(v, "v", (B, H, Dv))
        per_token = log_decay.dim() == 2
        gp = c.ptr(log_decay, "log_decay", torch.float32, (B, H) if per_token else (H,))
        sp = c.ptr(slots, "slots", torch.int32, (B,))
        hp = c.ptr(state, "state", torch.float32, (pool, H, Dk, Dv))
        if out is None:
            out = c.new((B, H, Dv), torch.bfloat16)
        op = c.ptr(out, "out", torch.bfloat16, (B, H, Dv))
        a = LinearAttentionStepArgs(_STEP_SIZE, B, pool, G, H, Dk, Dv, qp, kp, vp, qs[:2], ks[:2], vs[:2], gp,
                                    per_token, sp, scale, hp, op)
        status = _library().ss2d_linear_attention_step(a, c.handle)
        if status:
            _check(status, "ss2d_linear_attention_step")
    return out


def check_workspace_status(workspace, stream=None):
    """Raises Ss2dError (SS2D_ERR_DEVICE) if a tensor-core kernel's bounded wait ran out in the last
    matmul_fp8 or linear_attention on `workspace` (ss2d_workspace_status).  Synchronises the stream."""
    with _Call(workspace, stream) as c:
        _check(_library().ss2d_workspace_status(workspace.data_ptr(), c.handle), "ss2d_workspace_status")
