"""The operators on the GPU at values where their arithmetic could leave its range or lose bits that it should keep."""
import math

import pytest
import torch

import selective_scan_02_b200 as ss
from tests import operator_reference as ref
from tests.operator_reference import BF16, U
from tests.test_gpu_operators import _attention_inputs, _check_norm, _gen, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("rows,d", [(6, 256), (400, 256), (400, 301), (400, 5120), (5, 96), (3, 2049)])
def test_rms_norm_small_rows_with_a_small_eps(rows, d):
    """Scales at their floor of 2^-100: groups of zeros, of values near it, zero rows."""
    x = 1e-9 * torch.randn(rows, d, device="cuda", generator=_gen(d))
    x[1, d // 2:] = 0
    x[2] *= 1e-4
    w = torch.randn(d, device="cuda", generator=_gen(d + 1))
    w[:min(d, 128)] = 0
    w[128:130] = 1e-31
    for eps in (0.0, 1e-30, 1e-20, 1e-18, 1e-17):
        if eps:
            x[0] = 0
        for out in ("e4m3", "f32"):
            got = ss.rms_norm(x, w, eps=eps, out_dtype=torch.float8_e4m3fn if out == "e4m3" else torch.float32)
            assert torch.isfinite((got[0] if out == "e4m3" else got).float()).all()
            _check_norm(x, w, None, out, got, float(torch.tensor(eps, dtype=torch.float32)))


@pytest.mark.parametrize("rows,d", [(4, 512), (500, 1304), (500, 1301)])
def test_rms_norm_scales_are_rounded_once(rows, d):
    """Rows of plus and minus one have a norm of one: y is the weight, and a scale is a quotient, rounded once.  (CUDA's
    reciprocal root is within 2 units in the last place: 4 U of y.)"""
    x = torch.randint(0, 2, (rows, d), device="cuda", generator=_gen(1)).float() * 2 - 1
    w = torch.randn(d, device="cuda", generator=_gen(2))
    unit = ss.rms_norm(x, torch.ones_like(w), eps=0.0, out_dtype=torch.float32).abs()
    assert (unit == unit[0, 0]).all() and abs(unit[0, 0].item() - 1) <= 4 * U
    y = (unit[0, 0] * w).abs()
    q, s = ss.rms_norm(x, w, eps=0.0, out_dtype=torch.float8_e4m3fn)
    want = (torch.nn.functional.pad(y, (0, -d % 128)).view(-1, 128).amax(-1).double() / 448).float()
    assert (s == want).all()
    t = y.double() / want.double().repeat_interleave(128)[:d]
    step = torch.exp2(torch.floor(torch.log2(t.clamp_min(2.0 ** -6))) - 3)
    assert ((q.double().abs() - t).abs() <= step / 2 + 3 * U * t).all()
    assert (torch.signbit(q.float()) == torch.signbit(x * w)).all()


# ---- linear attention ------------------------------------------------------------------------------------


@pytest.mark.parametrize("shape", [(2, 700, 1, 2, 64, 40), (2, 8, 1, 2, 16, 24), (1, 6000, 1, 2, 128, 96), (20, 700, 2, 8, 64, 64),
                                   (30, 300, 1, 6, 24, 32)])
def test_a_nan_in_a_decay_reaches_no_token_before_its_own(shape):
    """Whole heads, token by token, segments, cut heads, the longest first: of the head and sequence of a NaN in log_decay, the
    outputs from its token on and the state are not finite; all else is what the definition gives without it."""
    B, L, G, H, Dk, Dv = shape
    q, k, v, gates, scale, h0 = _attention_inputs(shape, 401, True, True, True)
    n = torch.full((B,), L, device="cuda", dtype=torch.int32) if B == 30 else None
    clean, clean_last = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, lengths=n, return_last_state=True)
    for at in sorted({0, 5, L // 2, L - 1}):
        bad = gates.clone()
        bad[-1, at, -1] = math.nan
        out, last = ss.linear_attention(q, k, v, bad, scale=scale, h0=h0, lengths=n, return_last_state=True)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[-1, at:, -1] = True
        assert not out[hit].isfinite().any() and not last[-1, -1].isfinite().any()
        other = torch.ones(B, H, dtype=torch.bool, device="cuda")
        other[-1, -1] = False
        assert torch.equal(out.transpose(1, 2)[other], clean.transpose(1, 2)[other]) and torch.equal(last[other], clean_last[other])
        if at:
            head = [t[-1:, :at] for t in (q[:, :, -1:], k[:, :, -1:], v[:, :, -1:], gates[:, :, -1:])]
            want, _, size, _ = ref.linear_attention(*head, scale, h0[-1:, -1:])
            _within(out[-1:, :at, -1:], want, want.abs() * BF16 + size * (BF16 * 1.02) + 1e-30, "out")
    # one decay for each head
    bad = torch.full((H,), -0.1, device="cuda")
    bad[0] = math.nan
    out, last = ss.linear_attention(q, k, v, bad, scale=scale, h0=h0, lengths=n, return_last_state=True)
    assert not out[:, :, 0].isfinite().any() and not last[:, 0].isfinite().any()
    assert out[:, :, 1:].isfinite().all() and last[:, 1:].isfinite().all()
