"""The operators on the GPU at values where their arithmetic could leave its range or lose bits that it should keep."""
import math

import pytest
import torch

import selective_scan_02_b200 as ss
from tests import operator_reference as ref
from tests.operator_reference import BF16, U
from tests.test_gpu_operators import _attention_inputs, _check_attention, _check_norm, _gen, _matmul_inputs, _within

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


@pytest.mark.parametrize("batch,per_token", [(1, False), (1, True), (8, False), (8, True)])
def test_states_of_hundreds_of_chunks_keep_their_bits(batch, per_token):
    """300 chunks with slow decays, in one segment (a CTA for every head) and in several.

    A chunk's sum enters the state with two roundings of at most a half-step of it.  As independent errors, evenly spread over a
    step, 300 chunks that all count leave sqrt(600) U / sqrt(3) = 8.4e-7 of its norm, and the sums within a chunk little more:
    1e-6.  One bf16 part of w V less is 1e-5, and a chunk's decay rounded to one fp32 number 2e-6 to 5e-6 where it is slow."""
    L, D = 128 * 300, 64
    rates = torch.tensor([m * 2.0 ** -e for e in (15, 17, 19) for m in (1.0, 1.21, 1.37, 1.53, 1.71, 1.9)], device="cuda")
    H, g = len(rates), _gen(402)
    k = torch.randn(batch, L, 1, D, device="cuda", generator=g).bfloat16()
    v = torch.randn(batch, L, H, D, device="cuda", generator=g).bfloat16()
    gates = -rates if not per_token else (-rates).expand(batch, L, H).contiguous()
    ws = torch.empty(ss.linear_attention_workspace_size(batch, L, 1, H, D, D), dtype=torch.uint8, device="cuda")
    assert (ws.numel() > 256) == (batch == 1)  # segments' states
    _, last = ss.linear_attention(k, k, v, gates, return_last_state=True, workspace=ws)
    ss.check_workspace_status(ws)
    behind = torch.arange(L - 1, -1, -1, device="cuda", dtype=torch.float64)[:, None]
    for b in range(batch):
        for h in range(H):
            weight = torch.exp(-rates[h].double() * behind)
            want = k[b, :, 0].double().T @ (v[b, :, h].double() * weight)
            err = ((last[b, h].double() - want).norm() / want.norm()).item()
            assert err <= 1e-6, (b, h, err)


@pytest.mark.parametrize("m,n,k", [(4, 1024, 2048), (24, 520, 4096), (100, 300, 1104), (333, 1000, 1104), (1000, 1024, 4096)])
def test_products_keep_their_bits(m, n, k):
    """fp32 outputs.  A block's 128 products are exact, and their sum is cut off below about 2^-25 of its largest term in each
    of the MMAs' additions, or rounded; each block then takes one rounding: at most 64 blocks, sqrt(64) U / sqrt(3) = 2.8e-7 of
    the norm as independent errors, and half as much again for the blocks' sums: 5e-7."""
    a, sa, w, sw, bias = _matmul_inputs(m, n, k, m + n)
    want, _ = ref.matmul_fp8(a, sa, w, sw, bias)
    got = ss.matmul_fp8(a, sa, w, sw, bias=bias, out_dtype=torch.float32)
    assert ((got.double() - want).norm() / want.norm()).item() <= 5e-7


@pytest.mark.parametrize("shape", [(1, 390, 1, 2, 64, 64), (2, 700, 1, 2, 128, 96), (1, 6000, 1, 1, 64, 32)])
def test_runs_of_resets(shape):
    """Many tokens on end that reset the state, among slow decays: sums of thousands stand beside weights near one."""
    B, L, G, H, Dk, Dv = shape
    for value in (-math.inf, torch.finfo(torch.float32).min, -90.0):
        q, k, v, gates, scale, h0 = _attention_inputs(shape, 403, True, True, True)
        gates *= 0.05
        for lo, hi in ((3, 30), (45, 64), (100, 228), (300, 331)):
            gates[:, lo:hi] = value
        out, last = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True)
        _check_attention(q, k, v, gates, scale, h0, None, out, last)


@pytest.mark.parametrize("rows,d", [(3, 256), (400, 301), (400, 8192)])
def test_rms_norm_at_the_ends_of_its_range(rows, d):
    """Sums of squares just below 2^128, and with an eps of 0 rows of a root mean square of 2^-60."""
    x = torch.randn(rows, d, device="cuda", generator=_gen(d)).clamp_(-4, 4)
    w = torch.randn(d, device="cuda", generator=_gen(d + 1))
    x = x / x.square().mean(-1, keepdim=True).sqrt()
    for size, eps in ((0.99 * 2.0 ** 64 / d ** 0.5, 1e-6), (2.0 ** -60, 0.0)):
        for out in ("f32", "bf16", "e4m3"):
            dt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[out]
            _check_norm(x * size, w, None, out, ss.rms_norm(x * size, w, eps=eps, out_dtype=dt),
                        float(torch.tensor(eps, dtype=torch.float32)))


@pytest.mark.parametrize("heads,chunks", [(1, 600), (2, 600), (1, 2048)])
def test_states_of_many_segments_keep_their_bits(heads, chunks):
    """Over a hundred segments: bounds as for the chunks of one, the segments' sums being a tenth as many."""
    L, D = 128 * chunks, 64
    g = _gen(404)
    k = torch.randn(1, L, 1, D, device="cuda", generator=g).bfloat16()
    v = torch.randn(1, L, heads, D, device="cuda", generator=g).bfloat16()
    assert ss.linear_attention_workspace_size(1, L, 1, heads, D, D) > 60 * heads * D * D * 4
    behind = torch.arange(L - 1, -1, -1, device="cuda", dtype=torch.float64)[:, None]
    for rate in [m * 2.0 ** -e for e in (15, 17, 19, 21) for m in (1.0, 1.21, 1.53, 1.9)]:
        gates = torch.full((heads,), -rate, device="cuda")
        _, last = ss.linear_attention(k, k, v, gates, return_last_state=True)
        want = k[0, :, 0].double().T @ (v[0, :, -1].double() * torch.exp(gates[0].double() * behind))
        err = ((last[0, -1].double() - want).norm() / want.norm()).item()
        assert err <= 1e-6, (rate, err)
