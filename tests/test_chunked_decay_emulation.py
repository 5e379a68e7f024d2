"""The decay warp of the chunked linear attention on the host, against sums in 64 bits.

From a chunk's log decays it forms every factor that the other warps use: weights between two tokens as products or
exponents of a row's and a column's number, the decay from the chunk's start to a token, from a token to the chunk's end, and
across the chunk.  Each is compared with the exponential of the exact sum.  Its arguments are sums of at most 128 terms
in trees (a chain of 3 + 3 + 3 and one clamp and product each) of which the largest that still counts is below 2^8 (an
exponent of base 2 under -150 gives zero), so an argument is off by at most 32 half-steps of 2^8, and its factor
by ln 2 times that; the factors of two halves are multiplied.  A NaN must reach its own token and those behind it,
and no other."""
import os
import subprocess

import numpy as np
import pytest

from tests.emu_build import build_emulator
from tests.operator_reference import U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHUNK = 128

EXTRA = """
inline float emu_shfl(float v, int from)
{
    g_warp->slot[g_lane] = v;
    g_warp->bar.arrive_and_wait();
    const float r = g_warp->slot[from];
    g_warp->bar.arrive_and_wait();
    return r;
}
inline float __shfl_sync(unsigned, float v, int from) { return emu_shfl(v, from & 31); }
inline float __shfl_down_sync(unsigned, float v, int d, int width)
{
    const int at = g_lane % width + d;
    return emu_shfl(v, at < width ? g_lane + d : g_lane);
}
inline unsigned __ballot_sync(unsigned, bool p)
{
    emu_shfl(p ? 1.0f : 0.0f, 0);
    g_warp->slot[g_lane] = p ? 1.0f : 0.0f;
    g_warp->bar.arrive_and_wait();
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= (g_warp->slot[i] != 0.0f ? 1u : 0u) << i;
    g_warp->bar.arrive_and_wait();
    return r;
}
inline float __int_as_float(int v) { return __uint_as_float((uint32_t)v); }
inline int __ffs(unsigned v) { return __builtin_ffs((int)v); }
"""


@pytest.fixture(scope="module")
def emulator(tmp_path_factory):
    csrc = os.path.join(ROOT, "selective_scan_02_b200", "csrc")
    src = open(os.path.join(csrc, "linear_chunked.cu")).read()
    head = open(os.path.join(csrc, "linear_attention.h")).read()
    clamp = head[head.index("constexpr int kLaMaxDim"):head.index("// One call over whole sequences")]
    constants = src[src.index("constexpr int kLcChunk"):src.index("struct ChunkedArgs")]
    shapes = src[src.index("template <int DK, int DV, bool STATES = false>\nstruct Lc"):src.index("// kind::f16, fp32 accumulate")]
    first = "} else if (warp == 2) {"
    at = src.index(first) + len(first)
    warp = src[at:src.index("} else if (warp >= kLcWeight", at)]
    header = ('#pragma once\n#include "common_emu.h"\n' + EXTRA + "namespace ss2d {\n" + clamp + constants + shapes + "}\n")
    d = tmp_path_factory.mktemp("decay_emu")
    main = open(os.path.join(ROOT, "tests", "emu", "decay_emu_main.cpp")).read()
    lines = [line.split("//")[0].rstrip() for line in warp.splitlines()]
    body = " ".join(" _Pragma(\"GCC unroll 8\") " if line.strip() == "#pragma unroll" else line for line in lines)
    assert "DECAY_WARP" in main
    return build_emulator(d, header + "#define DECAY_WARP " + body + "\n", "decay_emu_main.cpp")


def _run(emulator, d, gates, first=0, end=None, states=False):
    gates = np.asarray(gates, np.float32)
    gates.tofile(os.path.join(d, "gates"))
    end = len(gates) if end is None else end
    r = subprocess.run([emulator, str(d), *map(str, (len(gates), first, end, int(states)))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    raw = np.fromfile(os.path.join(d, "decay"), np.float32)
    n = -(-(end - first) // CHUNK)
    fields = dict(cb=(CHUNK,), f=(CHUNK,), m=(4,), dm=(4, 4), e=(4,), keep=(), grow=())
    size = -(-(2 * CHUNK + 4 + 16 + 4 + 2) // 4) * 4
    out = []
    for c in range(n):
        part, at, got = raw[c * size:(c + 1) * size].astype(np.float64), 0, {}
        for name, shape in fields.items():
            k = int(np.prod(shape))
            got[name] = part[at:at + k].reshape(shape)
            at += k
        out.append(got)
    return out, float(raw[n * size])


def _factors(d):
    """What the other warps make of a chunk's factors: the weight of token j at token i, the decay from the chunk's start to
    i, and from j to its end."""
    blk = np.arange(CHUNK) // 32
    with np.errstate(over="ignore", invalid="ignore"):
        diag = np.exp2(d["cb"][:, None] - d["cb"][None, :])
        below = np.exp2(d["cb"][:, None] + d["dm"][blk][:, blk]) * d["f"][None, :]
        weight = np.where(blk[:, None] == blk[None, :], diag, below)
        return weight, np.exp2(d["cb"] + d["m"][blk]), d["f"] * d["e"][blk]


def _check(d, gates, nan_from=CHUNK):
    """gates: a chunk's, in 64 bits, with zeros behind the last token; tokens from nan_from on are NaN."""
    gates = np.maximum(gates, -128.0)
    c = np.cumsum(gates)
    i, j = np.arange(CHUNK)[:, None], np.arange(CHUNK)[None, :]
    weight, start, end = _factors(d)
    # of a reset in a block (an exponent of thousands in the sums), what is left of the tokens' own exponents
    worst = max(2.0 ** 8, np.abs(gates).sum() * 1.4426950408889634)
    tol = 32 * U * worst * np.log(2) * 2
    ok = i < nan_from
    lower = (j <= i) & ok
    want = np.exp(np.where(j <= i, c[:, None] - c[None, :], 0.0))
    assert (np.abs(weight - want)[lower] <= tol * want[lower] + 1e-37).all()
    keep = np.arange(CHUNK) < nan_from
    assert (np.abs(start - np.exp(c))[keep] <= tol * np.exp(c)[keep] + 1e-37).all()
    if nan_from == CHUNK:
        after = c[-1] - c
        assert (np.abs(end - np.exp(after)) <= tol * np.exp(after) + 1e-37).all()
        assert abs(d["keep"] + d["grow"] - np.exp(c[-1])) <= 16 * U * max(abs(c[-1]), 1e-30) + 1e-37
    else:
        assert np.isnan(start[~keep]).all() and np.isnan(weight[nan_from:, :]).all()
        assert np.isnan(end).any() or np.isnan(d["keep"] + d["grow"])  # the state behind


@pytest.mark.parametrize("rate", [1e-9, 1e-4, 0.01, 0.3, 5.0, 60.0])
@pytest.mark.parametrize("tokens", [1, 37, 128, 300])
def test_factors(emulator, tmp_path, tokens, rate):
    rng = np.random.default_rng(int(tokens * 7 + rate * 1000))
    gates = (-rate * rng.exponential(size=tokens)).astype(np.float32)
    got, _ = _run(emulator, tmp_path, gates)
    for c, d in enumerate(got):
        part = np.zeros(CHUNK)
        mine = gates[c * CHUNK:(c + 1) * CHUNK]
        part[:len(mine)] = mine
        _check(d, part)


@pytest.mark.parametrize("value", [-np.inf, np.finfo(np.float32).min, -1000.0])
def test_resets(emulator, tmp_path, value):
    rng = np.random.default_rng(5)
    for at in ([0], [31, 32], [5, 77, 127], list(range(20, 60)), list(range(128))):
        gates = (-0.1 * rng.exponential(size=CHUNK)).astype(np.float32)
        gates[at] = value
        _check(_run(emulator, tmp_path, gates)[0][0], gates.astype(np.float64))


@pytest.mark.parametrize("at", [[0], [1], [31], [32], [63, 70], [127], [5, 90], list(range(40, 128))])
def test_a_nan_reaches_no_token_before_its_own(emulator, tmp_path, at):
    rng = np.random.default_rng(at[0])
    gates = (-0.2 * rng.exponential(size=300)).astype(np.float32)
    bad = gates.copy()
    bad[np.array(at) + CHUNK] = np.nan  # in the second of three chunks
    got, _ = _run(emulator, tmp_path, bad)
    for c in (0, 2):
        part = np.zeros(CHUNK)
        mine = gates[c * CHUNK:(c + 1) * CHUNK]
        part[:len(mine)] = mine
        _check(got[c], part)
    part = gates[CHUNK:2 * CHUNK].astype(np.float64)
    part[at] = 0.0
    _check(got[1], part, at[0])
    if at[0]:  # behind the last token nothing is read
        got, _ = _run(emulator, tmp_path, bad, CHUNK, CHUNK + at[0])
        part = np.zeros(CHUNK)
        part[:at[0]] = gates[CHUNK:CHUNK + at[0]]
        _check(got[0], part)


@pytest.mark.parametrize("rate", [0.0, 1e-7, 2e-5, 3e-4, 0.002, 0.3])
def test_a_segment_s_decay(emulator, tmp_path, rate):
    """Of a slow one, the decay less 1, whose roundings are of its own size."""
    rng = np.random.default_rng(9)
    gates = (-rate * rng.exponential(size=1000)).astype(np.float32)
    _, decay = _run(emulator, tmp_path, gates, 128, 900, states=True)
    total = gates[128:900].astype(np.float64).sum()
    if np.signbit(np.float32(decay)):
        assert total >= -0.36 and abs(decay - np.expm1(total)) <= 64 * U * abs(total) + 1e-45
    else:
        assert total <= -0.34 and abs(decay - np.exp(total)) <= 64 * U * max(1, -total) * np.exp(total) + 2.0 ** -126  # (fp32's least)
