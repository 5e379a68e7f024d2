"""The operators on the GPU at values where their arithmetic could leave its range or lose bits that it should keep."""
import pytest
import torch

import selective_scan_02_b200 as ss
from tests.operator_reference import U
from tests.test_gpu_operators import _check_norm, _gen

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
