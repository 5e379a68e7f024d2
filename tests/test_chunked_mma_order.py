"""The order of the chunked linear attention's tensor-core instructions, checked without a GPU.

Two tcgen05.mma of one thread are ordered by the instruction set only where they have the same accumulator and the
same shape.  Any other two that touch the same columns of tensor memory (a write over a write, over a read of the
A operand, or the other way round) need a commit behind the first and a wait for that commit before the
second.  The branches of linear_chunked.cu's kernel that issue MMAs are compiled for the host and print what they
issue; every pair is checked.  A wait for an arrival that other warps make only behind a commit (the state's warps free a
buffer that they read after its commit, for instance) counts as a wait for that commit."""
import os
import re
import subprocess

import pytest

from tests.emu_build import build_emulator

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "selective_scan_02_b200", "csrc", "linear_chunked.cu")

# what another warp arrives at, and the commit that it has waited for by then
BEHIND = {"kOutFree": "kOutDone", "kInterFree": "kInterDone", "kDeltaFree": "kDeltaDone", "kProbsReady": "kScoresDone"}


def _between(src, first, last):
    at = src.index(first) + len(first)
    return src[at:src.index(last, at)]


@pytest.fixture(scope="module")
def emulator(tmp_path_factory):
    src = open(SOURCE).read()
    constants = src[src.index("constexpr int kLcChunk"):src.index("struct ChunkedArgs")]
    shapes = src[src.index("template <int DK, int DV, bool STATES = false>\nstruct Lc"):src.index("__device__ __forceinline__ uint32_t lc_pack")]
    scores = _between(src, "} else if (warp == 1 && !STATES) {", "} else if (warp == 3) {")
    state = _between(src, "} else if (warp == 3) {", "} else if (warp == 2) {")
    header = ("#pragma once\nnamespace ss2d {\n" + constants + shapes + "}\n")
    main = open(os.path.join(ROOT, "tests", "emu", "chunked_mma_main.cpp")).read()
    d = tmp_path_factory.mktemp("mma_order")
    exe = build_emulator(d, header + "#define ISSUE_SCORES\n#define ISSUE_STATE\n", "chunked_mma_main.cpp")
    # the branches are statements, with commas and comments of their own: they go in as text
    main = main.replace("        ISSUE_SCORES\n", scores).replace("        ISSUE_STATE\n", state)
    path = os.path.join(d, "main.cpp")
    with open(path, "w") as f:
        f.write(main)
    with open(os.path.join(d, "kernel_emu.h"), "w") as f:
        f.write(header)
    r = subprocess.run(["g++", "-std=c++20", "-O1", "-w", "-I", str(d), "-o", exe, path], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def _trace(exe, dk, dv, states, chunks, ready, warp):
    r = subprocess.run([exe, *map(str, (dk, dv, int(states), chunks, ready, warp))], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return [line.split() for line in r.stdout.splitlines()]


def _overlap(a, na, b, nb):
    return na > 0 and nb > 0 and a < b + nb and b < a + na


def _unordered(trace):
    """Pairs of MMAs that touch the same columns in no order that the instruction set gives."""
    bars = {int(t[2]): t[1] for t in trace if t[0] == "bar"}
    slots, deltas = next((int(t[1]), int(t[2])) for t in trace if t[0] == "rings")
    size = {"kScoresDone": 2, "kProbsReady": 2, "kWeightsReady": 2, "kWeightsFree": 2, "kDeltaDone": deltas, "kDeltaFree": deltas}
    size |= {n: slots for n in bars.values() if re.fullmatch(r"k[KQV](Free|Full|Checked)", n)}

    def name(bar):
        first = max(b for b in bars if b <= bar)
        assert bar - first < size.get(bars[first], 1)
        return bars[first], bar - first

    commits, waits, mmas = {}, {}, []  # of each barrier: places in the trace
    for at, t in enumerate(trace):
        if t[0] == "commit":
            commits.setdefault(name(int(t[1])), []).append(at)
        elif t[0] == "wait":
            which, i = name(int(t[1]))
            waits.setdefault((which, i), []).append((at, int(t[2])))
        elif t[0] == "mma":
            mmas.append((at, *map(int, t[1:])))
    # for each commit, the first wait that proves it done: the n-th commit of a barrier completes its n-th phase, whose
    # parity is n & 1; a wait for that parity behind it, before the phase after it, is a wait for it.  A barrier of
    # other warps passes the first time without any (a parity of 1), and then follows the commits one by one.
    proven = []
    for (which, i), places in commits.items():
        for n, at in enumerate(places):
            after = [w for w, parity in waits.get((which, i), []) if w > at and parity == n & 1]
            if after:
                proven.append((at, min(after)))
        for other, of in BEHIND.items():
            if of != which:
                continue
            behind = waits.get((other, i), [])
            passes_first = bool(behind) and behind[0][1] == 1  # "free" before it was ever taken
            for n, at in enumerate(places):
                if n + passes_first < len(behind):
                    proven.append((at, behind[n + passes_first][0]))
    bad = []
    for y, (ay, dy, ny, ry, rny, _, shape_y) in enumerate(mmas):
        for ax, dx, nx, rx, rnx, _, shape_x in mmas[:y]:
            if not (_overlap(dx, nx, dy, ny) or _overlap(dx, nx, ry, rny) or _overlap(rx, rnx, dy, ny)):
                continue
            if (dx, shape_x) == (dy, shape_y) and not _overlap(dx, nx, ry, rny) and not _overlap(rx, rnx, dy, ny):
                continue
            if not any(ax < c and w < ay for c, w in proven):
                bad.append((ax, ay))
    return bad


@pytest.mark.parametrize("ready", [0, 1, 2])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [32, 64])
def test_scores_and_outputs(emulator, dk, dv, ready):
    """The scores of a chunk replace those that the P V of two chunks before reads its P from."""
    for chunks in (1, 2, 3, 7):
        trace = _trace(emulator, dk, dv, False, chunks, ready, 1)
        assert sum(t[0] == "mma" for t in trace) == chunks * (dk // 16 + 8)
        assert not _unordered(trace)


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [32, 64])
def test_state_and_its_queries(emulator, dk, dv, states):
    """The parts of K^T (w V) that share columns."""
    for chunks in (1, 2, 5):
        trace = _trace(emulator, dk, dv, states, chunks, 1, 3)
        assert any(t[0] == "mma" for t in trace) and not _unordered(trace)


def test_the_check_sees_a_missing_wait():
    bars = [["bar", "kOutDone", "0"], ["bar", "kOutFree", "1"], ["rings", "2", "1"]]
    first, second = ["mma", "0", "64", "0", "0", "1", "7"], ["mma", "32", "64", "0", "0", "1", "7"]
    assert _unordered(bars + [first, ["commit", "0"], second])
    assert _unordered(bars + [first, ["wait", "0", "0"], ["commit", "0"], second])
    assert not _unordered(bars + [first, ["commit", "0"], ["wait", "0", "0"], second])
    assert not _unordered(bars + [["wait", "1", "1"], first, ["commit", "0"], ["wait", "1", "0"], second])
    assert not _unordered(bars + [first, ["mma", "0", "64", "0", "0", "1", "7"]])
    assert _unordered(bars + [first, ["mma", "0", "32", "0", "0", "1", "5"]])
