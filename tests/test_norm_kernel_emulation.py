"""rms_norm.cu's kernel on the host, against the definition in 64 bits, without a GPU.

The kernel's source, and the rule by which ss2d_rms_norm takes an instance of it, are compiled for the CPU with
tests/emu/: one std::thread per CUDA thread, warp shuffles and __syncthreads on barriers, the launcher's grid, under
AddressSanitizer and UBSan.  Widths span the instances, one row and several in a CTA, odd widths, cut groups.

Bounds count roundings of half a step each: the squares' sum is at most 32 + 64 additions in a chain, halved by the
root; then the root and three products.  CUDA's float to e4m3 is modelled from its definition (nearest, ties to even,
values above 448 become 448, NaN stays)."""
import os
import subprocess

import numpy as np
import pytest

from selective_scan_02_b200.inputs import bf16_bits, round_bf16
from tests.emu_build import build_emulator
from tests.operator_reference import BF16, E4M3, E4M3_TINY, U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF, F8 = range(3)

EXTRA = """
struct uint4 { unsigned x, y, z, w; };
inline uint4 make_uint4(unsigned a, unsigned b, unsigned c, unsigned d) { return {a, b, c, d}; }
inline uint2 make_uint2(unsigned a, unsigned b) { return {a, b}; }
inline void grid_wait() {}
inline void grid_next() {}
inline float rsqrtf(float x) { return (float)(1.0 / std::sqrt((double)x)); }
inline uint16_t emu_bf16(float f)
{
    uint32_t u = __float_as_uint(f);
    if (f != f) return 0x7fff;
    u += 0x7FFFu + ((u >> 16) & 1u);
    return (uint16_t)(u >> 16);
}
struct __nv_bfloat162 { uint16_t x, y; };
inline __nv_bfloat162 __floats2bfloat162_rn(float a, float b) { return {emu_bf16(a), emu_bf16(b)}; }
inline __nv_bfloat16 __float2bfloat16_rn(float f) { __nv_bfloat16 b; b.v = emu_bf16(f); return b; }
enum { __NV_SATFINITE, __NV_E4M3 };
inline uint8_t __nv_cvt_float_to_fp8(float f, int, int)
{
    if (f != f) return 0x7f;
    const uint8_t sign = std::signbit(f) ? 0x80 : 0;
    double t = std::min(std::fabs((double)f), 448.0);
    int e = std::max((int)std::floor(std::log2(std::max(t, 1e-300))), -6);
    double m = std::nearbyint(t / std::ldexp(1.0, e - 3));  // eighths of the binade; ties to even
    if (m >= 16) { m = 8; ++e; }
    if (m < 8) return sign | (uint8_t)m;  // below 2^-6
    return sign | (uint8_t)((e + 7) << 3 | ((int)m - 8));
}
inline uint16_t __nv_cvt_float2_to_fp8x2(float2 f, int s, int k)
{
    return (uint16_t)(__nv_cvt_float_to_fp8(f.x, s, k) | __nv_cvt_float_to_fp8(f.y, s, k) << 8);
}
enum { SS2D_F32, SS2D_BF16, SS2D_E4M3 };
"""


@pytest.fixture(scope="module")
def emulator(tmp_path_factory):
    src = open(os.path.join(ROOT, "selective_scan_02_b200", "csrc", "rms_norm.cu")).read()
    body = src[src.index("constexpr int kRnGroup"):src.index("cudaError_t rms_launch_types")]
    body = body[:body.rindex("template <")]
    shared = "__shared__ float part[kThreads / 32];"
    assert shared in body
    body = body.replace(shared, "float *const part = reinterpret_cast<float *>(g_warp->smem);")
    at = src.index("    if (D <= 8)\n")
    dispatch = src[at:src.index(";", src.index("    else\n", at)) + 1]
    launch = """
template <int TPR, int NV>
int rms_launch(const RmsArgs &a, int)
{
    constexpr int kThreads = TPR > kRnThreads ? TPR : kRnThreads;
    const unsigned grid = (unsigned)((a.rows + kThreads / TPR - 1) / (kThreads / TPR));
    auto run = [&](auto kernel) { emu_grid(grid, 1, kThreads, 128, [&] { kernel(a); }); return 0; };
    // the types' combinations that the tests use
    auto types = [&](auto vec) {
        constexpr bool V = decltype(vec)::value;
        if (!a.residual) return a.x_bf16 ? run(rms_norm_kernel<TPR, NV, V, true, kRnNone>) : 1;
        if (a.x_bf16) return a.res_bf16 ? 1 : run(rms_norm_kernel<TPR, NV, V, true, kRnF32>);
        return a.res_bf16 ? run(rms_norm_kernel<TPR, NV, V, false, kRnBf16>) : 1;
    };
    if (a.D % 8 == 0) return types(std::true_type{});
    return types(std::false_type{});
}
"""
    header = '#pragma once\n#include "common_emu.h"\n' + EXTRA + "namespace ss2d {\n" + body + launch + "}\n"
    d = tmp_path_factory.mktemp("norm_emu")
    return build_emulator(d, header + "#define DISPATCH " + " ".join(
        line.split("//")[0].strip() for line in dispatch.splitlines()) + "\n", "norm_emu_main.cpp")


def _e4m3(bits):
    b = bits.astype(np.int64)
    sign, e, m = np.where(b & 0x80, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((b & 0x7F) == 0x7F, np.nan, sign * v)


def _run(emulator, d, x, w, res, xt, rt, yt, eps, many):
    rows, D = x.shape
    (bf16_bits(x) if xt == BF else x).tofile(os.path.join(d, "x"))
    w.tofile(os.path.join(d, "weight"))
    if res is not None:
        (bf16_bits(res) if rt == BF else res).tofile(os.path.join(d, "residual"))
    code = 0 if res is None else 2 if rt == BF else 1
    r = subprocess.run([emulator, str(d), *map(str, (rows, D, int(xt == BF), code, yt, eps, int(many)))], capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]

    def read(name, t):
        raw = np.fromfile(os.path.join(d, name), {F32: np.float32, BF: np.uint16, F8: np.uint8}[t])
        return (raw.astype(np.uint32) << 16).view(np.float32) if t == BF else raw

    y = read("y", yt).reshape(rows, D)
    out = None if res is None else read("residual_out", rt).reshape(rows, D)
    if yt != F8:
        return y, None, out
    return _e4m3(y), np.fromfile(os.path.join(d, "scales"), np.float32).reshape(rows, -1), out


def _definition(x, w, res, eps):
    r = x.astype(np.float64) + (0 if res is None else res)
    with np.errstate(all="ignore"):
        return r / np.sqrt((r * r).mean(1, keepdims=True) + float(np.float32(eps))) * w.astype(np.float64), r


def _check(got, x, w, res, rt, yt, eps):
    q, s, out = got
    y, r = _definition(x, w, res, eps)
    slack = np.abs(y) * (64 * U) + 1e-40
    if yt == F8:
        D = x.shape[1]
        pad = np.pad(np.abs(y), ((0, 0), (0, -D % 128))).reshape(len(y), -1, 128).max(-1)
        want = np.maximum(pad / 448, 2.0 ** -100)
        assert (np.abs(s - want) <= want * (66 * U)).all()
        step = np.repeat(s.astype(np.float64), 128, 1)[:, :D]
        err, bound = np.abs(q * step - y), slack + np.abs(y) * E4M3 * (1 + 1e-5) + step * E4M3_TINY
    else:
        err, bound = np.abs(q - y), slack + np.abs(y) * (BF16 if yt == BF else U) * (1 + 1e-4)
    assert (err <= bound).all(), (err / bound).max()
    if res is not None:
        assert (np.abs(out - r) <= np.abs(r) * ((BF16 if rt == BF else 0) + U) * (1 + 1e-4) + 1e-40).all()


@pytest.mark.parametrize("rows,D,many", [(5, 1, False), (300, 7, False), (3, 16, True), (9, 33, True), (130, 41, False), (9, 64, True), (5, 129, False),
                                         (3, 256, True), (1, 400, False), (20, 384, True), (5, 333, True), (3, 720, True),
                                         (3, 1001, True), (2, 1301, True), (2, 2560, True), (1, 4100, True), (1, 4096, False)])
def test_widths(emulator, tmp_path, rows, D, many):
    rng = np.random.default_rng(rows * 10000 + D)
    for yt, xt, rt in ((F8, BF, F32), (BF, F32, BF), (F32, BF, None), (F8, F32, BF)):
        x = rng.standard_normal((rows, D)).astype(np.float32)
        x = round_bf16(x) if xt == BF else x
        w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
        res = None
        if rt is not None:
            res = (4 * rng.standard_normal((rows, D))).astype(np.float32)
            res = round_bf16(res) if rt == BF else res
        _check(_run(emulator, tmp_path, x, w, res, xt, rt, yt, 1e-5, many), x, w, res, rt, yt, 1e-5)


@pytest.mark.parametrize("D", [256, 301, 96])
def test_small_rows_with_a_small_eps(emulator, tmp_path, D):
    """Scales at their floor of 2^-100, which a norm's reciprocal of 2^28 and above takes beyond fp32 when the two are
    multiplied first: groups of zeros, of values near it and of none such, in rows that are small or zero."""
    rng = np.random.default_rng(D)
    for eps in (0.0, 1e-30, 1e-20, 1e-18, 1e-17):
        x = (1e-9 * rng.standard_normal((6, D))).astype(np.float32)
        x[1, D // 2:] = 0
        x[2] *= np.float32(1e-4)
        w = rng.standard_normal(D).astype(np.float32)
        w[:min(D, 128)] = 0             # a group whose values are all zero
        w[128:130] = 1e-31
        if eps:
            x[3] = 0
        res = np.zeros_like(x)
        x[4, -8:], x[5] = 1e-12, 1e-13
        for yt, rt in ((F8, BF), (F32, BF)):
            got = _run(emulator, tmp_path, x, w, res, F32, rt, yt, eps, True)
            assert np.isfinite(got[0]).all(), eps
            _check(got, x, w, res, rt, yt, eps)


def test_scales_are_rounded_once(emulator, tmp_path):
    """Rows of plus and minus one have a norm of one, so that y is the weight itself: the scale is the quotient of its group's
    maximum and 448, rounded once, and no column is further from its value than the rounding to e4m3 of a quotient that is
    itself within a step of fp32."""
    rng = np.random.default_rng(3)
    for D, many in ((512, True), (1301, True)):
        x = rng.choice(np.array([-1, 1], np.float32), (4, D))
        w = rng.standard_normal(D).astype(np.float32)
        q, s, _ = _run(emulator, tmp_path, x, w, None, BF, None, F8, 0.0, many)
        amax = np.pad(np.abs(w), (0, -D % 128)).reshape(-1, 128).max(-1)
        want = (amax.astype(np.float64) / 448).astype(np.float32)
        assert (s == want).all()
        t = np.abs(x * w / np.repeat(want, 128)[:D].astype(np.float64))
        unit = 2.0 ** (np.floor(np.log2(np.maximum(t, 2.0 ** -6))) - 3)
        assert (np.abs(np.abs(q) - t) <= unit / 2 + 3 * U * t).all()
