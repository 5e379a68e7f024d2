"""The operators' stream argument: every call of a layer on a stream that is not the current one, with outputs allocated by the
calls and given to them, against the same calls on the current stream."""
import pytest
import torch

import selective_scan_02_b200 as ss
from tests.test_gpu_operators import _attention_inputs, _gen, _Layer, _matmul_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _same(got, want):
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def _on(s):
    """Order a stream behind the current one's work, and back."""
    s.wait_stream(torch.cuda.current_stream())
    return s


@pytest.mark.parametrize("L", [7, 150])
def test_a_layer_on_a_given_stream(L):
    layer, d = _Layer(), 256
    x = torch.randn(3, L, d, device="cuda", generator=_gen(501)).bfloat16()
    res = torch.randn(3, L, d, device="cuda", generator=_gen(502))
    row, row_res = x[:, 0].contiguous(), res[:, 0].contiguous()
    want = [t.clone() for t in layer.prompt(x, res)]
    state = want[2].clone()
    want_row = [t.clone() for t in layer.step(row, row_res, state)]
    G, H, dk, dv = layer.sizes
    for given in (False, True):
        s = torch.cuda.Stream()
        out = torch.zeros(3, L, H, dv, device="cuda", dtype=torch.bfloat16) if given else None
        _on(s)
        q, k, v, r = layer._qkv(x, res, stream=s)
        o, after = ss.linear_attention(q, k, v, layer.gates, scale=dk ** -0.5, return_last_state=True, out=out, stream=s)
        assert not given or o is out
        y = layer._out(o, stream=s)
        got_row = layer.step(row, row_res, after, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        _same((y, r), want[:2])
        _same(got_row, want_row)
        assert torch.equal(after, state)


@pytest.mark.parametrize("shape", [(2, 6, 1, 2, 32, 40), (3, 300, 2, 4, 64, 64), (1, 6000, 1, 2, 128, 96), (20, 700, 2, 8, 64, 64)])
def test_given_outputs_and_workspaces_on_a_given_stream(shape):
    q, k, v, gates, scale, h0 = _attention_inputs(shape, 503, True, True, True)
    B, L, G, H, Dk, Dv = shape
    want = [t.clone() for t in ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True)]
    s = torch.cuda.Stream()
    out, last = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.full((ss.linear_attention_workspace_size(*shape),), 255, dtype=torch.uint8, device="cuda")
    got = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, out=out, h_last=last, workspace=ws, stream=_on(s))
    assert got[0] is out and got[1] is last
    ss.check_workspace_status(ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _same(got, want)
    # allocated by the call, and used on the current stream behind it while the other stream goes on allocating
    kept = []
    for _ in range(8):
        got = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True, stream=_on(s))
        torch.cuda.current_stream().wait_stream(s)
        kept.append([t + 0 for t in got])
        del got
    for got in kept:
        _same(got, want)
    row = [t[:, 0] for t in (q, k, v)] + [gates[:, 0].contiguous()]
    states = [h0.clone(), h0.clone()]
    want = ss.linear_attention_step(*row, states[0], scale=scale)
    into = torch.zeros_like(want)
    got = ss.linear_attention_step(*row, states[1], scale=scale, out=into, stream=_on(s))
    torch.cuda.current_stream().wait_stream(s)
    assert got is into
    _same((got, states[1]), (want, states[0]))


def test_products_and_norms_on_a_given_stream():
    a, sa, w, sw, bias = _matmul_inputs(70, 300, 1104, 504)
    want = ss.matmul_fp8(a, sa, w, sw, bias=bias)
    s = torch.cuda.Stream()
    out, ws = torch.zeros_like(want), torch.zeros(ss.matmul_fp8_workspace_size(70, 300, 1104), dtype=torch.uint8, device="cuda")
    assert ss.matmul_fp8(a, sa, w, sw, bias=bias, out=out, workspace=ws, stream=_on(s)) is out
    again = ss.matmul_fp8(a, sa, w, sw, bias=bias, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _same((out, again), (want, want))
    x = torch.randn(9, 333, device="cuda", generator=_gen(505)).bfloat16()
    weight = torch.randn(333, device="cuda", generator=_gen(506))
    want = ss.rms_norm(x, weight, residual=x, out_dtype=torch.float32)
    y, r = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    got = ss.rms_norm(x, weight, residual=x, y=y, residual_out=r, stream=_on(s))
    torch.cuda.current_stream().wait_stream(s)
    assert got[0] is y and got[1] is r
    _same(got, want)


def test_a_stream_of_another_kind_is_refused():
    x, w = torch.zeros(2, 128, device="cuda"), torch.ones(128, device="cuda")
    with pytest.raises(ValueError):
        ss.rms_norm([1.0], w, stream=torch.cuda.current_stream())
    with pytest.raises(ValueError):
        ss.rms_norm(x.cpu(), w, stream=torch.cuda.Stream())
