"""Slices of longer arrays as the arguments that are read one number at a time: the values of aligned copies."""
import pytest
import torch

import selective_scan_02_b200 as ss
from tests.test_gpu_operators import _attention_inputs, _gen, _matmul_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _slice(t, by):
    """t's values, `by` elements into a longer array."""
    pool = torch.zeros(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = pool[by:by + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16
    return out


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("m,n,k", [(3, 200, 272), (20, 130, 400), (70, 136, 1104), (300, 1001, 208)])
def test_matmul_scales_and_bias(m, n, k, by):
    a, sa, w, sw, bias = _matmul_inputs(m, n, k, m + by)
    want = ss.matmul_fp8(a, sa, w, sw, bias=bias)
    assert torch.equal(ss.matmul_fp8(a, _slice(sa, by), w, _slice(sw, by), bias=_slice(bias, by)), want)


@pytest.mark.parametrize("d", [96, 301, 4096])
def test_norm_scales(d):
    x = torch.randn(7, d, device="cuda", generator=_gen(d))
    w = torch.ones(d, device="cuda")
    y, s = ss.rms_norm(x, w, out_dtype=torch.float8_e4m3fn)
    into = _slice(torch.zeros_like(s), 3)
    again, got = ss.rms_norm(x, w, out_dtype=torch.float8_e4m3fn, scales=into)
    assert got is into and torch.equal(into, s) and torch.equal(again.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("shape", [(5, 7, 1, 2, 16, 24), (5, 300, 2, 4, 64, 64), (30, 300, 1, 6, 24, 32), (3, 5000, 1, 1, 24, 40)])
def test_lengths_and_slots(shape):
    B, L = shape[:2]
    q, k, v, gates, scale, h0 = _attention_inputs(shape, 91, True, True, True)
    n = torch.randint(0, L + 1, (B + 1,), device="cuda", generator=_gen(3), dtype=torch.int32)
    outs = [torch.zeros_like(v, memory_format=torch.contiguous_format) for _ in range(2)]
    got = [ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, lengths=m, return_last_state=True, out=o)[1]
           for m, o in zip((n[1:], n[1:].clone()), outs)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(got[0], got[1])
    slots = torch.randperm(B + 1, device="cuda", generator=_gen(4)).to(torch.int32)
    states = [torch.cat([h0, h0[:1]]).contiguous() for _ in range(2)]
    row = [t[:, 0] for t in (q, k, v)] + [gates[:, 0].contiguous()]
    outs = [ss.linear_attention_step(*row, s, slots=at, scale=scale) for s, at in zip(states, (slots[1:], slots[1:].clone()))]
    assert torch.equal(outs[0], outs[1]) and torch.equal(states[0], states[1])
