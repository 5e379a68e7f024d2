"""Definitions in 64 bits of the operators of a linear-attention layer, token by token and block by
block, and the rounding bounds that their kernels are held to."""
import torch

U = 2.0 ** -24        # half a step of fp32, relative
BF16 = 2.0 ** -8      # of bf16
E4M3 = 2.0 ** -4      # of e4m3
E4M3_TINY = 2.0 ** -10  # half a step of e4m3's subnormal numbers, absolute


def rms_norm(x, weight, residual, eps):
    """(y, r) in fp64."""
    r = x.double() if residual is None else x.double() + residual.double()
    return r / (r.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double(), r


def dequantise(q, scales, block=128):
    """The values (fp64) that e4m3 rows with a scale for each 128 columns stand for."""
    d = q.shape[-1]
    return q.double() * scales.double().repeat_interleave(block, dim=-1)[..., :d]


def matmul_fp8(a, a_scales, w, w_scales, bias):
    """(product, the same of absolute values) in fp64."""
    n = w.shape[0]
    av = dequantise(a, a_scales)
    wv = dequantise(w, w_scales.repeat_interleave(128, dim=0)[:n])
    c, size = av @ wv.T, av.abs() @ wv.abs().T
    if bias is not None:
        c, size = c + bias.double(), size + bias.double().abs()
    return c, size


def linear_attention(q, k, v, log_decay, scale, h0=None, lengths=None):
    """(out, h_last, out's terms, h_last's terms): the last two are the sums of the absolute values of
    what out and h_last are sums of.  Rows of out behind a sequence's end are zero."""
    B, L, G, Dk = q.shape
    H, Dv = v.shape[2:]
    q, k = (t.double().repeat_interleave(H // G, dim=2) for t in (q, k))
    v = v.double()
    g = log_decay.double().expand(B, L, H)
    S = torch.zeros(B, H, Dk, Dv, dtype=torch.float64, device=q.device) if h0 is None else h0.double().clone()
    A = S.abs()
    out = torch.zeros(B, L, H, Dv, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    n = torch.full((B,), L, device=q.device) if lengths is None else lengths.clamp(0, L)
    for t in range(L):
        on = (t < n)[:, None, None, None]
        decay = g[:, t].exp()[..., None, None]
        kv = k[:, t, :, :, None] * v[:, t, :, None, :]
        S = torch.where(on, S * decay + kv, S)
        A = torch.where(on, A * decay + kv.abs(), A)
        out[:, t] = torch.where(on[..., 0], (q[:, t, :, :, None] * S).sum(2) * scale, 0.0)
        size[:, t] = torch.where(on[..., 0], (q[:, t, :, :, None].abs() * A).sum(2) * abs(scale), 0.0)
    return out, S, size, A
