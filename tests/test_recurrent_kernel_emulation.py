"""Linear attention's CUDA-core kernels run on the host, against the definition in 64 bits, without a GPU.

linear_recurrent_kernel of selective_scan_02_b200/csrc/linear_recurrent.cu (short prompts, and steps
on a pool of states) and linear_carry_kernel of linear_chunked.cu (the states of a long sequence's
segments, added up) are compiled for the CPU with tests/emu/: one std::thread per CUDA thread,
__syncthreads on a per-CTA barrier, the launchers' grids, under AddressSanitizer and UBSan.  Shapes span
widths that end inside a CTA's 32 columns, lengths of none, one and all tokens, slots outside the
pool, and rows that name one slot again.

Bounds: an output is rounded to bf16 once and otherwise, like a state, a sum of fp32 products: a state of n tokens is
within 4 n + 8 half-steps of its terms' absolute sum, an output within Dk more."""
import os
import subprocess

import numpy as np
import pytest
import torch

from selective_scan_02_b200.inputs import bf16_bits, round_bf16
from tests import operator_reference as ref
from tests.emu_build import build_emulator
from tests.operator_reference import BF16, U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_scan_02_b200", "csrc")

EXTRA = """
inline uint2 make_uint2(unsigned a, unsigned b) { return {a, b}; }
inline void grid_wait() {}
inline void grid_next() {}
inline __nv_bfloat16 __float2bfloat16_rn(float f)
{
    uint32_t u = __float_as_uint(f);
    u += 0x7FFFu + ((u >> 16) & 1u);
    __nv_bfloat16 b;
    b.v = (uint16_t)(u >> 16);
    return b;
}
template <class T> inline T __ldcs(const T *p) { return *p; }
template <class T> inline void __stcs(T *p, T v) { *p = v; }
inline void atomicMin(int *p, int v)
{
    std::atomic_ref<int> r(*p);
    int old = r.load();
    while (v < old && !r.compare_exchange_weak(old, v)) {}
}
"""


def _piece(name, first, last):
    src = open(os.path.join(CSRC, name)).read()
    return src[src.index(first):src.index(last)]


@pytest.fixture(scope="module")
def emulator(tmp_path_factory):
    args = _piece("linear_attention.h", "constexpr int kLaMaxDim", "// Token by token.")
    body = _piece("linear_recurrent.cu", "constexpr int kLrThreads", "template <bool STEP>\ncudaError_t launch_rows")
    shared = ("    __shared__ float sq[kLaMaxDim], sk[kLaMaxDim];\n"
              "    __shared__ float part[kLrThreads / 32][kLrCols];\n"
              "    __shared__ int next_row;\n")
    assert shared in body
    body = body.replace(shared, "    Shared &sh = *reinterpret_cast<Shared *>(g_warp->smem);\n"
                                "    auto &sq = sh.sq, &sk = sh.sk;\n    auto &part = sh.part;\n    int &next_row = sh.next_row;\n")
    carry = _piece("linear_chunked.cu", "constexpr int kLcCarry = 8", "// Tensor map over")
    assert "__shared__" not in body + carry
    constants, kernel = body.split("// STEP: the tokens", 1)
    shared = ("struct Shared { alignas(16) float sq[kLaMaxDim], sk[kLaMaxDim], part[kLrThreads / 32][kLrCols]; int next_row, any; };\n"
              "constexpr size_t kEmuShared = sizeof(Shared);\n"
              # every thread's value, by way of the CTA's shared memory
              "inline bool __syncthreads_or(bool v)\n{\n    int &any = reinterpret_cast<Shared *>(g_warp->smem)->any;\n"
              "    if (threadIdx.x == 0) any = 0;\n    __syncthreads();\n"
              "    if (v) std::atomic_ref<int>(any).store(1);\n    __syncthreads();\n    const bool r = any != 0;\n"
              "    __syncthreads();\n    return r;\n}\n")
    header = ('#pragma once\n#include "common_emu.h"\n' + EXTRA + "namespace ss2d {\n" + args + constants + shared +
              "// STEP: the tokens" + kernel + carry + "}  // namespace ss2d\n")
    return build_emulator(tmp_path_factory.mktemp("recurrent_emu"), header, "recurrent_emu_main.cpp")


def _run(emulator, d, mode, B, L, G, H, Dk, Dv, per_token, pool, **tensors):
    for name, t in tensors.items():
        (bf16_bits(t) if name in ("q", "k", "v", "out") else t).tofile(os.path.join(d, name))
    r = subprocess.run([emulator, str(d), *[str(int(x)) for x in (mode, B, L, G, H, Dk, Dv, per_token, pool)]],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    state = torch.from_numpy(np.fromfile(os.path.join(d, "state"), np.float32))
    if mode == 4:
        return state
    out = (np.fromfile(os.path.join(d, "out"), np.uint16).astype(np.uint32) << 16).view(np.float32)
    return torch.from_numpy(out).view(B, L, H, Dv), state.view(-1, H, Dk, Dv)


def _inputs(seed, B, L, G, H, Dk, Dv, per_token, states):
    rng = np.random.default_rng(seed)
    t = {n: round_bf16(rng.standard_normal(s).astype(np.float32))
         for n, s in (("q", (B, L, G, Dk)), ("k", (B, L, G, Dk)), ("v", (B, L, H, Dv)))}
    t["gates"] = -np.exp(rng.uniform(-6, 1, (B, L, H) if per_token else (H,))).astype(np.float32)
    t["gates"].reshape(-1)[0] = -np.inf
    t["state"] = rng.standard_normal((states, H, Dk, Dv)).astype(np.float32)
    t["out"] = np.full((B, L, H, Dv), 3.0, np.float32)
    return t


def _close(got, want, size, terms, n, out=False):
    bound = size * n * U + (want.abs() * BF16 * (1 + 2 * n * U) if out else 0) + 1e-30
    assert ((got.double() - want).abs() <= bound).all(), ((got.double() - want).abs() / bound).max()


@pytest.mark.parametrize("B,L,G,H,Dk,Dv,per_token", [(1, 1, 1, 1, 8, 8, False), (4, 8, 1, 3, 24, 40, True),
                                                     (2, 5, 2, 2, 128, 128, False), (1, 3, 1, 2, 56, 8, True)])
@pytest.mark.parametrize("lengths", [False, True])
def test_prompts(emulator, tmp_path, B, L, G, H, Dk, Dv, per_token, lengths):
    t = _inputs(B + L, B, L, G, H, Dk, Dv, per_token, B)
    n = None
    if lengths:
        n = np.array([L, 0, 1, L + 9][:B] if B > 1 else [L], np.int32)
    out, state = _run(emulator, tmp_path, int(lengths), B, L, G, H, Dk, Dv, per_token, 0, **t,
                      **({"lengths": n} if lengths else {}))
    w = {k: torch.from_numpy(x) for k, x in t.items()}
    n = None if n is None else torch.from_numpy(n).clamp(0, L)
    want, S, size, terms = ref.linear_attention(w["q"], w["k"], w["v"], w["gates"], 0.5, w["state"], n)
    behind = torch.arange(L) >= (torch.full((B,), L) if n is None else n)[:, None]
    assert (out[behind] == 3).all()
    keep = ~behind
    _close(out[keep], want[keep], size[keep], None, 4 * L + 8 + Dk, out=True)
    _close(state, S, terms, None, 4 * L + 8)


@pytest.mark.parametrize("G,H,Dk,Dv,per_token", [(1, 2, 16, 24, True), (2, 2, 128, 64, False)])
def test_steps(emulator, tmp_path, G, H, Dk, Dv, per_token):
    pool, slots = 5, np.array([4, 1, 4, -1, 4, 5, 0], np.int32)  # rows of slot 4 follow one another
    B = len(slots)
    t = _inputs(Dk, B, 1, G, H, Dk, Dv, per_token, pool)
    out, state = _run(emulator, tmp_path, 3, B, 1, G, H, Dk, Dv, per_token, pool, **t, slots=slots)
    w = {k: torch.from_numpy(x) for k, x in t.items()}
    S, A = w["state"].double().clone(), w["state"].double().abs()
    for b, slot in enumerate(slots):
        if not 0 <= slot < pool:
            assert (out[b] == 3).all()
            continue
        gates = w["gates"][b:b + 1] if per_token else w["gates"]
        args = (w["q"][b:b + 1], w["k"][b:b + 1], w["v"][b:b + 1], gates, 0.5)
        want, S1, _, _ = ref.linear_attention(*args, S[slot:slot + 1])
        _, A1, size, _ = ref.linear_attention(*(x.abs() for x in args[:3]), gates, 0.5, A[slot:slot + 1])
        S[slot], A[slot] = S1[0], A1[0]
        _close(out[b], want[0], size[0], None, 4 * 3 + 8 + Dk, out=True)
    _close(state, S, A, None, 4 * 3 + 8)
    # without slots, row b has state b
    t = _inputs(Dv, 3, 1, G, H, Dk, Dv, per_token, 4)
    out, state = _run(emulator, tmp_path, 2, 3, 1, G, H, Dk, Dv, per_token, 4, **t)
    w = {k: torch.from_numpy(x) for k, x in t.items()}
    want, S, size, terms = ref.linear_attention(w["q"], w["k"], w["v"], w["gates"], 0.5, w["state"][:3])
    _close(out, want, size, None, 12 + Dk, out=True)
    _close(state[:3], S, terms, None, 12)
    assert torch.equal(state[3], w["state"][3])


@pytest.mark.parametrize("heads,segments,Dk,Dv", [(1, 2, 8, 8), (3, 8, 24, 40), (2, 9, 16, 128), (1, 30, 64, 8)])
def test_carry(emulator, tmp_path, heads, segments, Dk, Dv):
    rng = np.random.default_rng(segments)
    states = rng.standard_normal((heads, segments, Dk, Dv)).astype(np.float32)
    decays = rng.uniform(0, 1, (heads, segments)).astype(np.float32)
    got = _run(emulator, tmp_path, 4, heads, segments, 1, heads, Dk, Dv, False, 0, state=states, gates=decays)
    want, size = states.astype(np.float64), np.abs(states.astype(np.float64))
    for i in range(1, segments):
        want[:, i] += want[:, i - 1] * decays[:, i, None, None]
        size[:, i] += size[:, i - 1] * decays[:, i, None, None]
    err = np.abs(got.numpy().reshape(states.shape) - want)
    assert (err <= size * segments * U).all()


def test_carry_of_slow_decays(emulator, tmp_path):
    """Decays near 1 come less 1: the state behind 140 segments keeps its bits (each takes two roundings of a half-step; as
    independent errors sqrt(280) U / sqrt(3) of the norm, 5.8e-7), where rounded decays would lose 140 half-steps of their own."""
    rng = np.random.default_rng(4)
    heads, segments, D = 2, 140, 16
    states = rng.standard_normal((heads, segments, D, D)).astype(np.float32)
    less = -(2.0 ** -rng.uniform(9, 24, (heads, 1)) * np.ones((1, segments)))
    less[1, ::7] = 0.0  # no decay at all
    less = np.copysign(less, -1.0).astype(np.float32)
    got = _run(emulator, tmp_path, 4, heads, segments, 1, heads, D, D, False, 0, state=states, gates=less)
    want = states.astype(np.float64)
    for i in range(1, segments):
        want[:, i] += want[:, i - 1] * (1.0 + less[:, i, None, None].astype(np.float64))
    last, exact = got.numpy().reshape(states.shape)[:, -1], want[:, -1]
    err = np.linalg.norm(last - exact, axis=(1, 2)) / np.linalg.norm(exact, axis=(1, 2))
    assert (err <= 6e-7).all(), err
