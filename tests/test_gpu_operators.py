"""GPU parity of the operators of a linear-attention layer against their definitions in 64 bits.

Bounds count roundings (operator_reference.py gives half a step of each type):
  - fp32 sums of n terms are within n half-steps of the terms' absolute sum; the kernels add in trees
    or tensor-core blocks, so fewer apply, and each test says which count it takes;
  - an output rounded once adds half a step of its type;
  - linear attention multiplies bf16 by bf16 on the tensor cores: the decayed scores and the carried
    state are rounded to bf16 for that (one half-step of the terms' absolute sum each), while the state
    itself is summed from v times its decay in three bf16 parts, which leave 2^-24 of each term."""
import math

import pytest
import torch

import selective_scan_02_b200 as ss
from tests import operator_reference as ref
from tests.operator_reference import BF16, E4M3, E4M3_TINY, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _within(got, want, bound, what=""):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), what
    worst = ((got - want).abs() / bound.clamp_min(1e-300)).max().item()
    assert worst <= 1.0, (what, worst)


# ---- rms_norm --------------------------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 5), (7, 8), (5, 41), (33, 96), (2, 127), (9, 128), (6, 200), (4, 768), (17, 1000), (3, 1001),
               (5, 2048), (4, 4096), (1, 4100), (2, 8192), (3, 12288), (2, 32768), (1, 32767)]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _norm_bounds(x, w, res, eps):
    """y and its bound before the output's rounding: the squares' sum (at most 32 + 64 additions in a chain,
    halved by the root), the root and three products."""
    y, r = ref.rms_norm(x, w, res, eps)
    return y, r, y.abs() * (64 * U) + 1e-40


def _check_norm(x, w, res, out, got, eps):
    y, r, slack = _norm_bounds(x, w, res, eps)
    got = got if isinstance(got, tuple) else (got,)
    assert len(got) == 1 + (out == "e4m3") + (res is not None)
    if out == "e4m3":
        q, s = got[:2]
        d = x.shape[-1]
        pad = torch.nn.functional.pad(y, (0, -d % 128)).unflatten(-1, (-1, 128))
        want = (pad.abs().amax(-1) / 448).clamp_min(2.0 ** -100)
        _within(s, want, want * (66 * U), "scales")
        step = s.double().repeat_interleave(128, dim=-1)[..., :d]
        _within(ref.dequantise(q, s), y, slack + y.abs() * E4M3 * (1 + 1e-5) + step * E4M3_TINY, "e4m3")
    else:
        _within(got[0], y, slack + y.abs() * (BF16 if out == "bf16" else U) * (1 + 1e-4), "y")
    if res is not None:
        _within(got[-1], r, r.abs() * ((BF16 if res.dtype == torch.bfloat16 else 0) + U) * (1 + 1e-4) + 1e-40, "residual")


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("rows,d", NORM_SHAPES)
def test_rms_norm(rows, d, out):
    for i, (xt, rt) in enumerate([("bf16", "f32"), ("f32", "bf16"), ("bf16", None), ("f32", None)]):
        g = _gen(rows * 100000 + d * 10 + i)
        x = torch.randn(rows, d, device="cuda", generator=g).to(TYPES[xt])
        w = 1 + 0.3 * torch.randn(d, device="cuda", generator=g)
        res = None if rt is None else (4 * torch.randn(rows, d, device="cuda", generator=g)).to(TYPES[rt])
        _check_norm(x, w, res, out, ss.rms_norm(x, w, residual=res, eps=1e-5, out_dtype=TYPES[out]), 1e-5)


def test_rms_norm_many_rows():
    g = _gen(4)
    x = torch.randn(70001, 32, device="cuda", generator=g).bfloat16()
    w = torch.ones(32, device="cuda")
    _check_norm(x, w, None, "bf16", ss.rms_norm(x, w, eps=1e-6), 1e-6)


@pytest.mark.parametrize("d", [1, 2, 7, 8, 9, 16, 17, 24, 31, 33, 40, 64, 65, 100, 128, 129, 201, 264, 333, 384,
                               512, 640, 701, 1000, 1301, 1536, 2048, 2049, 2560, 4096, 5001, 5120, 8192, 10000, 12285, 16384,
                               20000, 20001, 24576, 32768])
def test_rms_norm_widths_of_many_rows(d):
    """A row more than two for each SM: other splits of a row than the few rows' above."""
    g = _gen(d)
    x = torch.randn(297, d, device="cuda", generator=g).bfloat16()
    w = 1 + 0.3 * torch.randn(d, device="cuda", generator=g)
    for out, res in (("e4m3", torch.randn(297, d, device="cuda", generator=g)), ("bf16", None),
                     ("f32", torch.randn(297, d, device="cuda", generator=g).bfloat16())):
        _check_norm(x, w, res, out, ss.rms_norm(x, w, residual=res, eps=1e-5, out_dtype=TYPES[out]), 1e-5)
        _check_norm(x.float(), w, res, out, ss.rms_norm(x.float(), w, residual=res, eps=1e-5, out_dtype=TYPES[out]), 1e-5)


def test_rms_norm_in_place_and_leading_dimensions():
    g = _gen(5)
    x = torch.randn(2, 3, 320, device="cuda", generator=g).bfloat16()
    w = torch.randn(320, device="cuda", generator=g)
    res = torch.randn(2, 3, 320, device="cuda", generator=g)
    before = res.clone()
    y, s, r = ss.rms_norm(x, w, residual=res, residual_out=res, out_dtype=torch.float8_e4m3fn)
    assert r is res and y.shape == x.shape and s.shape == (2, 3, 3)
    _check_norm(x, w, before, "e4m3", (y, s, res), 1e-6)


def test_rms_norm_zero_huge_and_nan_rows():
    x = torch.ones(5, 256, device="cuda")
    x[1] = 0
    x[2, 128:] = 0
    x[3] *= 1e15
    x[4, 7] = float("nan")
    w = torch.ones(256, device="cuda")
    q, s = ss.rms_norm(x, w, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(q[1].float(), torch.zeros(256, device="cuda")) and (s[1] == 2.0 ** -100).all()
    assert (q[2, :128].float() == 448).all() and (q[2, 128:].float() == 0).all()
    _within(ref.dequantise(q[3], s[3]), torch.ones(256, device="cuda"), torch.full((256,), E4M3, device="cuda"))
    assert torch.isnan(q[4].float()).all() and not torch.isnan(q[:4].float()).any()
    # with eps 0 a zero row has no norm: 0 / 0
    assert torch.isnan(ss.rms_norm(x[1:2], w, eps=0.0)).all()


# ---- matmul_fp8 ------------------------------------------------------------------------------------------

MATMUL_SHAPES = [(1, 1, 16), (1, 128, 128), (2, 129, 144), (5, 300, 208), (16, 256, 512), (17, 1000, 1104), (33, 64, 4096),
                 (64, 4096, 2048), (65, 136, 272), (127, 255, 128), (128, 128, 128), (129, 257, 384), (200, 2056, 1360),
                 (300, 100, 8192), (512, 512, 1024), (1000, 1001, 496), (2049, 640, 256), (4, 6144, 2048)]


def _e4m3(shape, g, spread=90.0):
    return (spread * torch.randn(shape, device="cuda", generator=g)).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _matmul_inputs(m, n, k, seed):
    g = _gen(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    a, w = _e4m3((m, k), g), _e4m3((n, k), g)
    sa = torch.exp(torch.randn(m, kb, device="cuda", generator=g)) / 90
    sw = torch.exp(torch.randn(nb, kb, device="cuda", generator=g)) / 90
    return a, sa, w, sw, torch.randn(n, device="cuda", generator=g)


def _check_matmul(got, a, sa, w, sw, bias):
    want, size = ref.matmul_fp8(a, sa, w, sw, bias)
    # a block of 128 products is exact in each of the tensor core's additions but for their truncation (one
    # step, two half-steps, for each of at most 128), then one product and one addition for each block
    n = 2 * 128 + 3 * sa.shape[-1] + 2
    # the typical sum of roundings of either sign is far below their number
    _within(got, want, size * (n * U) + (want.abs() * BF16 if got.dtype == torch.bfloat16 else 0.0) + 1e-30, "product")
    rel = ((got.double() - want).norm() / want.norm()).item()
    assert rel <= (BF16 if got.dtype == torch.bfloat16 else 1e-5), rel


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", MATMUL_SHAPES)
def test_matmul_fp8(m, n, k, out_dtype):
    a, sa, w, sw, bias = _matmul_inputs(m, n, k, m * 7 + n * 3 + k)
    for b in (None, bias):
        ws = torch.full((ss.matmul_fp8_workspace_size(m, n, k),), 255, dtype=torch.uint8, device="cuda")
        got = ss.matmul_fp8(a, sa, w, sw, bias=b, out_dtype=out_dtype, workspace=ws)
        ss.check_workspace_status(ws)
        _check_matmul(got, a, sa, w, sw, b)


def test_matmul_fp8_writes_its_output_alone():
    for m, n, k in ((3, 130, 160), (140, 70, 400), (1, 8, 16)):
        a, sa, w, sw, _ = _matmul_inputs(m, n, k, 3)
        for dt in (torch.bfloat16, torch.float32):
            pool = torch.full((m * n + 64,), 7.0, dtype=dt, device="cuda")
            out = pool[32:32 + m * n].view(m, n)
            ss.matmul_fp8(a, sa, w, sw, out=out)
            _check_matmul(out, a, sa, w, sw, None)
            assert (pool[:32] == 7).all() and (pool[32 + m * n:] == 7).all()


def test_matmul_fp8_leading_dimensions_and_nan():
    a, sa, w, sw, _ = _matmul_inputs(6, 40, 144, 9)
    got = ss.matmul_fp8(a.view(2, 3, 144), sa.view(2, 3, 2), w, sw)
    assert got.shape == (2, 3, 40)
    _check_matmul(got.view(6, 40), a, sa, w, sw, None)
    bad = a.clone()
    bad.view(torch.uint8)[4, 10] = 0x7F
    nan = torch.isnan(ss.matmul_fp8(bad, sa, w, sw))
    assert nan[4].all() and not nan[:4].any() and not nan[5:].any()


# ---- linear attention ------------------------------------------------------------------------------------

# B, L, G, H, Dk, Dv
ATTENTION_SHAPES = [(1, 1, 1, 1, 8, 8), (2, 3, 1, 2, 16, 24), (3, 64, 2, 2, 64, 64), (1, 127, 1, 3, 40, 56),
                    (2, 128, 2, 4, 128, 128), (1, 129, 1, 1, 128, 64), (2, 200, 2, 6, 64, 128), (1, 300, 5, 5, 72, 104),
                    (2, 513, 1, 2, 128, 128), (1, 1025, 1, 1, 64, 32), (5, 196, 1, 6, 64, 32), (1, 2000, 2, 2, 128, 120)]


def _attention_inputs(shape, seed, per_token, h0, fused, lead=None):
    B, L, G, H, Dk, Dv = shape
    g = _gen(seed)
    lead = (B, L) if lead is None else lead
    widths = [G * Dk, G * Dk, H * Dv]
    if fused:
        parts = torch.randn(*lead, sum(widths), device="cuda", generator=g).bfloat16().split(widths, dim=-1)
    else:
        parts = [torch.randn(*lead, w, device="cuda", generator=g).bfloat16() for w in widths]
    q, k, v = (p.unflatten(-1, s) for p, s in zip(parts, [(G, Dk), (G, Dk), (H, Dv)]))
    if per_token:
        gates = -torch.exp(2.7 * torch.rand(H, device="cuda", generator=g)) * torch.nn.functional.softplus(
            torch.randn(*lead, H, device="cuda", generator=g) - 3)
    else:
        gates = torch.log1p(-torch.exp2(-2 - 7 * torch.rand(H, device="cuda", generator=g)))
    state = torch.randn(B, H, Dk, Dv, device="cuda", generator=g) if h0 else None
    return q, k, v, gates, Dk ** -0.5, state


def _check_attention(q, k, v, gates, scale, h0, lengths, out, h_last):
    want, S, size, terms = ref.linear_attention(q, k, v, gates, scale, h0, lengths)
    L = q.shape[1]
    # scores and carried state rounded to bf16, the output rounded to bf16, fp32 elsewhere
    _within(out, want, want.abs() * BF16 + size * (BF16 * 1.02) + 1e-30, "out")
    if want.norm() > 0:
        assert ((out.double() - want).norm() / want.norm()).item() <= BF16, "out"
    # three bf16 parts of each term, at most 128 truncated additions in a chunk, two roundings for each chunk
    n = 2 * 128 + 2 * math.ceil(L / 128) + 8
    _within(h_last, S, terms * (2.0 ** -24 + n * U) + 1e-30, "h_last")
    if S.norm() > 0:
        assert ((h_last.double() - S).norm() / S.norm()).item() <= 1e-5, "h_last"


@pytest.mark.parametrize("per_token,h0,fused", [(False, False, False), (True, True, True), (False, True, False),
                                                (True, False, True)])
@pytest.mark.parametrize("shape", ATTENTION_SHAPES)
def test_linear_attention(shape, per_token, h0, fused):
    q, k, v, gates, scale, state = _attention_inputs(shape, sum(shape), per_token, h0, fused)
    B, L, G, H, Dk, Dv = shape
    ws = torch.full((ss.linear_attention_workspace_size(*shape),), 255, dtype=torch.uint8, device="cuda")
    out, last = ss.linear_attention(q, k, v, gates, scale=scale, h0=state, return_last_state=True, workspace=ws)
    ss.check_workspace_status(ws)
    _check_attention(q, k, v, gates, scale, state, None, out, last)


@pytest.mark.parametrize("shape", [(5, 300, 2, 4, 64, 64), (6, 700, 1, 2, 128, 128), (4, 9, 1, 1, 16, 8)])
def test_linear_attention_lengths(shape):
    """Sequences of none, one, a tile's and other lengths; what lies behind them is NaN and stays unread, and
    the output's rows there stay as they were."""
    B, L, G, H, Dk, Dv = shape
    q, k, v, gates, scale, state = _attention_inputs(shape, 11, True, True, True)
    lengths = torch.tensor(([0, 1, L, 128, 129, L - 1] if L > 129 else [0, 1, L, 5, 2, 3])[:B], device="cuda",
                           dtype=torch.int32)
    pad = torch.arange(L, device="cuda") >= lengths[:, None]
    for t in (q, k, v):
        t[pad] = float("nan")
    gates[pad] = float("nan")
    out = torch.full((B, L, H, Dv), 3.0, device="cuda", dtype=torch.bfloat16)
    got, last = ss.linear_attention(q, k, v, gates, scale=scale, h0=state, lengths=lengths, return_last_state=True, out=out)
    assert got is out and (out[pad] == 3).all()
    clean = [torch.where(pad[..., None, None], torch.zeros_like(t), t) for t in (q, k, v)]
    g = torch.where(pad[..., None], torch.zeros_like(gates), gates)
    _check_attention(*clean, g, scale, state, lengths, torch.where(pad[..., None, None], torch.zeros_like(out), out), last)
    assert torch.equal(last[0], state[0])
    # lengths beyond L or below 0 are held within the range
    wild = torch.where(lengths == L, lengths + 1000, torch.where(lengths == 0, lengths - 7, lengths))
    out2, last2 = ss.linear_attention(q, k, v, gates, scale=scale, h0=state, lengths=wild, return_last_state=True,
                                      out=out.clone())
    assert torch.equal(out2, out) and torch.equal(last2, last)


def test_linear_attention_state_passing_and_in_place():
    """Pieces of a sequence, each continued from the state of the one before, replaced in place."""
    shape = (2, 421, 2, 4, 64, 96)
    q, k, v, gates, scale, state = _attention_inputs(shape, 12, True, True, False)
    h = state.clone()
    outs = []
    for lo, hi in ((0, 1), (1, 130), (130, 258), (258, 421)):
        o, got = ss.linear_attention(q[:, lo:hi], k[:, lo:hi], v[:, lo:hi], gates[:, lo:hi].contiguous(), scale=scale,
                                     h0=h, h_last=h)
        assert got is h
        outs.append(o)
    _check_attention(q, k, v, gates, scale, state, None, torch.cat(outs, 1), h)


@pytest.mark.parametrize("shape", [(20, 700, 2, 8, 64, 64), (40, 900, 1, 2, 24, 72), (19, 1300, 1, 16, 128, 24),
                                   (32, 650, 1, 5, 16, 16)])
def test_linear_attention_cut_units(shape):
    """A little more than one or two CTAs for each SM, so that the last heads are cut in two: sequences that end
    in either piece or at the cut, with the state replaced in place; and the same in a graph."""
    B, L, G, H, Dk, Dv = shape
    q, k, v, gates, scale, state = _attention_inputs(shape, 18, True, True, True)
    gates *= 0.1
    cut = (-(-L // 128) + 1) // 2 * 128
    lengths = torch.full((B,), L, device="cuda", dtype=torch.int32)
    lengths[-7:] = torch.tensor([L - 1, cut, cut + 1, cut - 1, 0, 1, L], device="cuda", dtype=torch.int32)
    ws = torch.full((ss.linear_attention_workspace_size(*shape),), 255, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 256  # the cut heads' states
    for n in (None, lengths):
        h, out = state.clone(), torch.zeros(B, L, H, Dv, device="cuda", dtype=torch.bfloat16)
        ss.linear_attention(q, k, v, gates, scale=scale, h0=h, h_last=h, lengths=n, out=out, workspace=ws)
        ss.check_workspace_status(ws)
        _check_attention(q, k, v, gates, scale, state, n, out, h)
    again, h2 = torch.zeros_like(out), state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.linear_attention(q, k, v, gates, scale=scale, h0=h2, h_last=h2, lengths=lengths, out=again, workspace=ws)
    for _ in range(3):
        h2.copy_(state)
        graph.replay()
        assert torch.equal(again, out) and torch.equal(h2, h)


@pytest.mark.parametrize("shape", [(1, 700, 1, 2, 128, 96), (2, 300, 1, 2, 64, 40), (1, 8, 1, 2, 16, 40),
                                   (1, 5000, 1, 1, 32, 24)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_linear_attention_not_finite(shape, value):
    """An infinity or a NaN reaches no token before its own, and of v no other column: all else is as without it."""
    B, L, G, H, Dk, Dv = shape
    q, k, v, gates, scale, state = _attention_inputs(shape, 17, True, True, False)
    clean, clean_last = ss.linear_attention(q, k, v, gates, scale=scale, h0=state, return_last_state=True)
    at = L // 2 + 1
    first = torch.arange(L, device="cuda") < at
    bad = v.clone()
    bad[-1, at, -1, [3, Dv - 1]] = value
    out, last = ss.linear_attention(q, k, bad, gates, scale=scale, h0=state, return_last_state=True)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[-1, at:, -1, [3, Dv - 1]] = True
    assert not out[hit].isfinite().any() and torch.equal(out[~hit], clean[~hit])
    hit = torch.zeros_like(last, dtype=torch.bool)
    hit[-1, -1, :, [3, Dv - 1]] = True
    assert not last[hit].isfinite().any() and torch.equal(last[~hit], clean_last[~hit])
    bad = k.clone()
    bad[-1, at, 0, 5] = value
    out, last = ss.linear_attention(q, bad, v, gates, scale=scale, h0=state, return_last_state=True)
    assert not out[-1, at:].isfinite().any() and torch.equal(out[:, first], clean[:, first])
    assert not last[-1, :, 5].isfinite().any()
    rest = [d for d in range(Dk) if d != 5]
    assert torch.equal(last[-1, :, rest], clean_last[-1, :, rest]) and torch.equal(last[:-1], clean_last[:-1])
    bad = q.clone()
    bad[-1, at, 0, 5] = value
    out, last = ss.linear_attention(bad, k, v, gates, scale=scale, h0=state, return_last_state=True)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[-1, at] = True
    assert not out[hit].isfinite().any() and torch.equal(out[~hit], clean[~hit]) and torch.equal(last, clean_last)


@pytest.mark.parametrize("shape", [(4, 4000, 1, 1, 128, 96), (4, 9000, 1, 1, 24, 40)])
def test_linear_attention_segments_ragged_and_in_place(shape):
    """Few heads, so that a sequence is cut into segments: lengths that end in the first, an inner and the last
    one, or before the first token, with the state replaced in place."""
    B, L, G, H, Dk, Dv = shape
    q, k, v, gates, scale, state = _attention_inputs(shape, 16, True, True, True)
    gates[:, 2000:2050:7] = -math.inf
    gates *= 0.02  # slow: what the segments carry counts
    lengths = torch.tensor([L, 2500, 0, 131], device="cuda", dtype=torch.int32)
    out = torch.zeros(B, L, H, Dv, device="cuda", dtype=torch.bfloat16)
    h = state.clone()
    ss.linear_attention(q, k, v, gates, scale=scale, h0=h, h_last=h, lengths=lengths, out=out)
    _check_attention(q, k, v, gates, scale, state, lengths, out, h)
    assert torch.equal(h[2], state[2])
    # without a state before and without the one behind
    ss.linear_attention(q, k, v, gates, scale=scale, lengths=lengths, out=out)
    want = ref.linear_attention(q, k, v, gates, scale, None, lengths)
    _within(out, want[0], want[0].abs() * BF16 + want[2] * (BF16 * 1.02) + 1e-30, "out")


def test_linear_attention_resets_and_no_decay():
    """Log decays of -infinity and of the type's lowest value reset the state; zero keeps all of it."""
    shape = (1, 390, 1, 2, 64, 64)
    for value in (-math.inf, torch.finfo(torch.float32).min, -1000.0):
        q, k, v, gates, scale, state = _attention_inputs(shape, 13, True, True, False)
        gates[:, [0, 1, 77, 127, 128, 200, 389]] = value
        out, last = ss.linear_attention(q, k, v, gates, scale=scale, h0=state, return_last_state=True)
        _check_attention(q, k, v, gates, scale, state, None, out, last)
    q, k, v, gates, scale, state = _attention_inputs(shape, 14, True, True, False)
    out, last = ss.linear_attention(q, k, v, torch.full_like(gates, -math.inf), scale=scale, h0=state,
                                    return_last_state=True)
    _check_attention(q, k, v, torch.full_like(gates, -math.inf), scale, state, None, out, last)
    none = torch.zeros(2, device="cuda")
    out, last = ss.linear_attention(q, k, v, none, scale=scale, h0=state, return_last_state=True)
    _check_attention(q, k, v, none, scale, state, None, out, last)


def test_linear_attention_strides():
    """Heads before tokens, every other token, padded rows: the same values as from dense tensors."""
    shape = (2, 260, 2, 2, 64, 64)
    q, k, v, gates, scale, _ = _attention_inputs(shape, 15, True, False, False)
    want, last = ss.linear_attention(q, k, v, gates, scale=scale, return_last_state=True)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    kt = torch.zeros(2, 520, 2, 64, device="cuda", dtype=torch.bfloat16)[:, ::2]
    kt.copy_(k)
    vt = torch.zeros(2, 260, 2, 72, device="cuda", dtype=torch.bfloat16)[..., :64]
    vt.copy_(v)
    out, got = ss.linear_attention(qt, kt, vt, gates, scale=scale, return_last_state=True)
    assert torch.equal(out, want) and torch.equal(got, last)


def test_linear_attention_refuses_views_it_cannot_read():
    q = torch.zeros(1, 8, 1, 64, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(1, device="cuda")
    with pytest.raises(ValueError):
        ss.linear_attention(q.transpose(1, 3), q.transpose(1, 3), q.transpose(1, 3), g)
    odd = torch.zeros(1, 8, 1, 68, device="cuda", dtype=torch.bfloat16)[..., :64]
    with pytest.raises(ss.Ss2dError):
        ss.linear_attention(odd, q, q, g)
    with pytest.raises(ss.Ss2dError):
        ss.linear_attention(q[:, :1].expand(1, 8, 1, 64), q, q, g)
    with pytest.raises(ValueError):
        ss.linear_attention(q.float(), q, q, g)
    with pytest.raises(ValueError):
        ss.linear_attention(q, q, q, g.double())


# ---- one token -------------------------------------------------------------------------------------------

# B, pool, G, H, Dk, Dv
STEP_SHAPES = [(1, 1, 1, 1, 8, 8), (3, 3, 1, 2, 16, 24), (2, 4, 2, 4, 128, 128), (7, 9, 1, 3, 40, 56), (33, 48, 8, 24, 64, 96),
               (130, 130, 1, 1, 64, 32), (300, 311, 1, 1, 8, 16)]


def _check_step(q, k, v, gates, scale, before, slots, out, after, kept):
    """Row by row: rows of one slot follow one another."""
    B, G, Dk = q.shape
    H = v.shape[1]
    S = before.double()
    A = S.abs()
    at = list(range(B)) if slots is None else slots.tolist()
    for b in range(B):
        if not 0 <= at[b] < before.shape[0]:
            assert torch.equal(out[b], kept[b])
            continue
        o, last, size, terms = ref.linear_attention(q[b][None, None], k[b][None, None], v[b][None, None],
                                                    (gates if gates.dim() == 1 else gates[b][None, None]), scale,
                                                    S[at[b]][None])
        S[at[b]] = last[0]
        A[at[b]] = torch.maximum(A[at[b]], terms[0])
        # one product and one addition for each element, the sum over Dk in a tree of at most 16 additions
        _within(out[b], o[0, 0], o[0, 0].abs() * BF16 + size[0, 0] * (24 * U) + 1e-30, "out")
    _within(after, S, A * (8 * B * U) + 1e-30, "state")


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("with_slots", [False, True])
@pytest.mark.parametrize("shape", STEP_SHAPES)
def test_linear_attention_step(shape, with_slots, per_token):
    B, pool, G, H, Dk, Dv = shape
    q, k, v, gates, scale, _ = _attention_inputs((B, 1, G, H, Dk, Dv), sum(shape), per_token, False, with_slots, lead=(B,))
    state = torch.randn(pool, H, Dk, Dv, device="cuda", generator=_gen(1))
    slots = None
    if with_slots:
        slots = torch.randperm(pool, device="cuda", generator=_gen(2))[:B].to(torch.int32)
        slots[::5] = -1
    before = state.clone()
    kept = torch.full((B, H, Dv), 2.0, device="cuda", dtype=torch.bfloat16)
    out = ss.linear_attention_step(q, k, v, gates, state, slots=slots, scale=scale, out=kept.clone())
    _check_step(q, k, v, gates, scale, before, slots, out, state, kept)


def test_linear_attention_step_rows_of_one_slot_and_wild_slots():
    B, pool, H, Dk, Dv = 150, 6, 2, 32, 40
    q, k, v, gates, scale, _ = _attention_inputs((B, 1, 1, H, Dk, Dv), 21, True, False, False, lead=(B,))
    state = torch.randn(pool, H, Dk, Dv, device="cuda", generator=_gen(3))
    slots = torch.randint(-2, pool + 2, (B,), device="cuda", generator=_gen(4), dtype=torch.int32)
    slots[0], slots[1] = torch.iinfo(torch.int32).min, torch.iinfo(torch.int32).max
    before = state.clone()
    kept = torch.full((B, H, Dv), 2.0, device="cuda", dtype=torch.bfloat16)
    out = ss.linear_attention_step(q, k, v, gates, state, slots=slots, scale=scale, out=kept.clone())
    _check_step(q, k, v, gates, scale, before, slots, out, state, kept)


# ---- offsets beyond 32 bits ------------------------------------------------------------------------------


def test_rms_norm_offsets_beyond_32_bits():
    rows, d = 2 ** 31 // 4096 + 300, 4096
    x = torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16)
    x[-200:] = torch.randn(200, d, device="cuda", generator=_gen(51)).bfloat16()
    w = torch.ones(d, device="cuda")
    y, s = ss.rms_norm(x, w, out_dtype=torch.float8_e4m3fn)
    _check_norm(x[-200:], w, None, "e4m3", (y[-200:], s[-200:]), 1e-6)
    assert (s[:-200] == 2.0 ** -100).all()


def test_matmul_fp8_offsets_beyond_32_bits():
    m, n, k = 2 ** 31 // 32768 + 200, 32768, 128
    a, sa, w, sw, _ = _matmul_inputs(m, n, k, 52)
    got = ss.matmul_fp8(a, sa, w, sw)
    _check_matmul(got[-150:], a[-150:], sa[-150:], w, sw, None)


def test_linear_attention_offsets_beyond_32_bits():
    """A reset near the end leaves little to compute for the definition."""
    B, L, H, D, tail = 1, 2 ** 31 // (256 * 64) + 500, 256, 64, 70
    g = _gen(53)
    q, k = (torch.randn(B, L, 1, 8, device="cuda", generator=g).bfloat16() for _ in range(2))
    v = torch.zeros(B, L, H, D, device="cuda", dtype=torch.bfloat16)
    v[:, -tail:] = torch.randn(B, tail, H, D, device="cuda", generator=g).bfloat16()
    gates = torch.full((B, L, H), -0.05, device="cuda")
    gates[:, -tail] = -math.inf
    out, last = ss.linear_attention(q, k, v, gates, return_last_state=True)
    _check_attention(q[:, -tail:], k[:, -tail:], v[:, -tail:], gates[:, -tail:], 1.0, None, None, out[:, -tail:], last)
    assert (out[:, :-tail] == 0).all()


def test_linear_attention_step_offsets_beyond_32_bits():
    H, D = 8, 128
    pool = 2 ** 31 // (H * D * D) + 50
    state = torch.zeros(pool, H, D, D, device="cuda")
    q, k, v, gates, scale, _ = _attention_inputs((3, 1, 1, H, D, D), 54, True, False, False, lead=(3,))
    slots = torch.tensor([pool - 1, 7, pool - 20], device="cuda", dtype=torch.int32)
    state[slots.long()] = torch.randn(3, H, D, D, device="cuda", generator=_gen(55))
    before = state[slots.long()].clone()
    kept = torch.zeros(3, H, D, device="cuda", dtype=torch.bfloat16)
    out = ss.linear_attention_step(q, k, v, gates, state, slots=slots, scale=scale)
    _check_step(q, k, v, gates, scale, before, None, out, state[slots.long()], kept)
    state[slots.long()] = 0
    assert not state.any()


# ---- together --------------------------------------------------------------------------------------------

def _quantise_weight(w):
    """e4m3 weights with a scale for each 128 x 128 block, as a user lays them out once."""
    n, k = w.shape
    pad = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128)).unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
    s = (pad.abs().amax((1, 3)) / 448).clamp_min(2.0 ** -100)
    q = (pad / s[:, None, :, None]).flatten(2).flatten(0, 1)[:n, :k].to(torch.float8_e4m3fn).contiguous()
    return q, s


class _Layer:
    """norm, q k v projection, linear attention, norm, output projection: one layer as it is served."""

    def __init__(self, d=256, H=4, G=2, dk=64, dv=64, seed=31):
        g = _gen(seed)
        self.sizes = (G, H, dk, dv)
        self.w1 = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
        self.w2 = 1 + 0.1 * torch.randn(H * dv, device="cuda", generator=g)
        self.win = _quantise_weight(torch.randn(2 * G * dk + H * dv, d, device="cuda", generator=g) / d ** 0.5)
        self.wout = _quantise_weight(torch.randn(d, H * dv, device="cuda", generator=g) / (H * dv) ** 0.5)
        self.gates = torch.log1p(-torch.exp2(-3 - torch.arange(H, device="cuda").float()))

    def _qkv(self, x, residual, **kw):
        G, H, dk, dv = self.sizes
        y, s, r = ss.rms_norm(x, self.w1, residual=residual, out_dtype=torch.float8_e4m3fn, **kw)
        qkv = ss.matmul_fp8(y, s, *self.win, **kw)
        q, k, v = qkv.split([G * dk, G * dk, H * dv], dim=-1)
        return q.unflatten(-1, (G, dk)), k.unflatten(-1, (G, dk)), v.unflatten(-1, (H, dv)), r

    def _out(self, o, **kw):
        y, s = ss.rms_norm(o.flatten(-2), self.w2, out_dtype=torch.float8_e4m3fn, **kw)
        return ss.matmul_fp8(y, s, *self.wout, **kw)

    def prompt(self, x, residual, lengths=None, h0=None, **kw):
        q, k, v, r = self._qkv(x, residual, **kw)
        o, state = ss.linear_attention(q, k, v, self.gates, scale=q.shape[-1] ** -0.5, lengths=lengths, h0=h0,
                                       return_last_state=True, out=torch.zeros_like(v, memory_format=torch.contiguous_format), **kw)
        return self._out(o, **kw), r, state

    def step(self, x, residual, state, **kw):
        q, k, v, r = self._qkv(x, residual, **kw)
        o = ss.linear_attention_step(q, k, v, self.gates, state, scale=q.shape[-1] ** -0.5, **kw)
        return self._out(o, **kw), r


def test_layer_prompt_then_tokens_is_the_whole_prompt():
    """A prompt and then single tokens give what the whole sequence as a prompt gives.  Both sides round the
    attention's output to bf16 from values that differ by the prompt's bf16 scores, one half-step or so, which
    the e4m3 rounding behind it turns into a step of e4m3 here and there: an element of the output is a sum of
    256 products, each off by at most a step (2 x 2^-4) of itself where that happens, in quadrature."""
    layer, B, L, n, d = _Layer(), 3, 160, 147, 256
    g = _gen(32)
    x = torch.randn(B, L, d, device="cuda", generator=g).bfloat16()
    res = torch.randn(B, L, d, device="cuda", generator=g)
    want, _, last = layer.prompt(x, res)
    _, _, state = layer.prompt(x[:, :n].contiguous(), res[:, :n].contiguous())
    for t in range(n, L):
        got, r = layer.step(x[:, t].contiguous(), res[:, t].contiguous(), state)
        diff = (got.double() - want[:, t].double()).norm() / want[:, t].double().norm()
        assert diff.item() <= 2 * E4M3, (t, diff.item())
    # the states differ by what the two sums' fp32 arithmetic does
    assert ((state - last).norm() / last.norm()).item() <= 1e-5


def test_layer_in_a_graph_on_two_streams():
    """The layer captured and replayed, with two captured graphs in flight at once on two streams."""
    layer, d = _Layer(), 256
    g = _gen(33)
    runs = []
    for i in range(2):
        x = torch.randn(2, 150, d, device="cuda", generator=g).bfloat16()
        res = torch.randn(2, 150, d, device="cuda", generator=g)
        eager = [t.clone() for t in layer.prompt(x, res)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            out = layer.prompt(x, res)
        runs.append((s, graph, out, eager, (x, res)))  # a replay reads its inputs again
    torch.cuda.synchronize()
    for _ in range(3):
        for s, graph, out, eager, _ in runs:
            with torch.cuda.stream(s):
                for t in out:
                    t.fill_(float("nan"))
                graph.replay()
        torch.cuda.synchronize()
        for s, graph, out, eager, _ in runs:
            for got, want in zip(out, eager):
                assert torch.equal(got, want)


def test_calls_on_several_streams_at_once():
    """Calls in flight together, of every kind of split: cut heads, segments, clusters, and the step."""
    calls, wanted = [], []
    for i, shape in enumerate([(20, 700, 2, 8, 64, 64), (1, 9000, 1, 2, 128, 96), (3, 500, 1, 2, 40, 24)]):
        q, k, v, gates, scale, state = _attention_inputs(shape, 70 + i, True, True, True)
        calls.append(lambda q=q, k=k, v=v, g=gates, s=state: ss.linear_attention(q, k, v, g, h0=s, return_last_state=True))
    for i, (m, n, k) in enumerate([(4, 4096, 2048), (100, 512, 4096), (700, 900, 1040)]):
        a, sa, w, sw, bias = _matmul_inputs(m, n, k, 80 + i)
        calls.append(lambda a=a, sa=sa, w=w, sw=sw, b=bias: (ss.matmul_fp8(a, sa, w, sw, bias=b),))
    q, k, v, gates, scale, state = _attention_inputs((30, 1, 4, 8, 128, 64), 90, True, True, False, lead=(30,))

    def step():
        s = state.clone()
        return ss.linear_attention_step(q, k, v, gates, s), s

    calls.append(step)
    wanted = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = []
        for s, call in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(call())
                got[-1] = call()
        torch.cuda.synchronize()
        for have, want in zip(got, wanted):
            assert all(torch.equal(x, y) for x, y in zip(have, want))


def test_layer_on_a_given_stream():
    layer, d = _Layer(), 256
    x = torch.randn(2, 40, d, device="cuda", generator=_gen(34)).bfloat16()
    res = torch.randn(2, 40, d, device="cuda", generator=_gen(35))
    want = layer.prompt(x, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, sc, r = ss.rms_norm(x, layer.w1, residual=res, out_dtype=torch.float8_e4m3fn, stream=s)
    qkv = ss.matmul_fp8(y, sc, *layer.win, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y2, sc2, r2 = ss.rms_norm(x, layer.w1, residual=res, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(qkv, ss.matmul_fp8(y2, sc2, *layer.win)) and torch.equal(r, r2)
    assert all(torch.isfinite(t.float()).all() for t in want)


def test_workspace_status_reports_the_error_word():
    """Every call clears the word; a word that is set says so, and the context stays usable."""
    a, sa, w, sw, _ = _matmul_inputs(4, 64, 128, 61)
    ws = torch.full((ss.matmul_fp8_workspace_size(4, 64, 128),), 255, dtype=torch.uint8, device="cuda")
    ss.matmul_fp8(a, sa, w, sw, workspace=ws)
    ss.check_workspace_status(ws)
    ws.view(torch.int32)[0] = 1
    with pytest.raises(ss.Ss2dError) as e:
        ss.check_workspace_status(ws)
    assert e.value.name == "SS2D_ERR_DEVICE"
    for L in (3, 200):  # token by token, and in chunks
        q, k, v, gates, scale, _ = _attention_inputs((1, L, 1, 1, 64, 64), 62, True, False, False)
        ws = torch.full((ss.linear_attention_workspace_size(1, L, 1, 1, 64, 64),), 255, dtype=torch.uint8, device="cuda")
        ss.linear_attention(q, k, v, gates, workspace=ws)
        ss.check_workspace_status(ws, stream=torch.cuda.current_stream())
    with pytest.raises(ss.Ss2dError):
        ss.matmul_fp8(a, sa, w, sw, workspace=ws[:16])


def test_wrong_arguments_are_refused():
    a, sa, w, sw, bias = _matmul_inputs(6, 40, 144, 63)
    for bad in (dict(a_scales=sa[:, :1].contiguous()), dict(w_scales=sw.double()), dict(w=w[:, :128].contiguous()),
                dict(bias=bias[:20]), dict(bias=bias.bfloat16()), dict(a_scales=sa.cpu()), dict(a=a.view(torch.uint8)),
                dict(out=torch.empty(6, 41, device="cuda")), dict(out_dtype=torch.float16)):
        args = dict(a=a, a_scales=sa, w=w, w_scales=sw)
        with pytest.raises(ValueError):
            ss.matmul_fp8(**(args | bad))
    with pytest.raises(ss.Ss2dError) as e:
        ss.matmul_fp8(a[:, :136].contiguous(), sa, w[:, :136].contiguous(), sw)
    assert e.value.name == "SS2D_ERR_UNSUPPORTED"
    x = torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)
    one = torch.ones(128, device="cuda")
    for bad in (dict(weight=one[:64]), dict(weight=one.bfloat16()), dict(residual=x.half()), dict(residual=x[:2]),
                dict(out_dtype=torch.float16), dict(scales=torch.empty(4, 1, device="cuda")), dict(x=x.t()),
                dict(residual_out=x), dict(x=x.half())):
        with pytest.raises(ValueError):
            ss.rms_norm(**(dict(x=x, weight=one) | bad))
    with pytest.raises(ss.Ss2dError):
        ss.rms_norm(x, one, y=x)
    with pytest.raises(ss.Ss2dError):
        ss.rms_norm(x[:0], one)
    with pytest.raises(ss.Ss2dError):
        ss.rms_norm(x, one, eps=-1.0)
    with pytest.raises(ss.Ss2dError) as e:
        ss.rms_norm(x.flatten()[1:-127].view(3, 128), one)
    assert e.value.name == "SS2D_ERR_MISALIGNED"
    q, k, v, gates, scale, state = _attention_inputs((2, 5, 1, 2, 16, 16), 64, False, True, False)
    for bad in (dict(k=k[:, :4]), dict(v=v.float()), dict(log_decay=gates[:1]), dict(log_decay=gates.view(1, 2)),
                dict(h0=state[:1]), dict(lengths=torch.zeros(2, device="cuda", dtype=torch.int64)),
                dict(lengths=torch.zeros(3, device="cuda", dtype=torch.int32)), dict(q=q[0])):
        with pytest.raises(ValueError):
            ss.linear_attention(**(dict(q=q, k=k, v=v, log_decay=gates) | bad))
    with pytest.raises(ss.Ss2dError):
        ss.linear_attention(q, k, v[:, :, :1].expand(2, 5, 2, 16), gates)
    row = dict(q=q[:, 0], k=k[:, 0], v=v[:, 0], log_decay=gates, state=state)
    for bad in (dict(state=state.bfloat16()), dict(state=state[..., :8]), dict(slots=torch.zeros(2, device="cuda")),
                dict(q=q), dict(state=state[0])):
        with pytest.raises(ValueError):
            ss.linear_attention_step(**(row | bad))
    with pytest.raises(ss.Ss2dError):
        ss.linear_attention_step(**(row | dict(state=state[:1])))  # fewer states than rows


def test_repeated_calls_are_identical():
    shape = (2, 1100, 1, 4, 128, 128)
    q, k, v, gates, scale, h0 = _attention_inputs(shape, 41, True, True, True)
    first = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True)
    a, sa, w, sw, bias = _matmul_inputs(70, 300, 2048, 42)
    c = ss.matmul_fp8(a, sa, w, sw, bias=bias)
    for _ in range(3):
        again = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True)
        assert all(torch.equal(s, t) for s, t in zip(first, again))
        assert torch.equal(c, ss.matmul_fp8(a, sa, w, sw, bias=bias))
