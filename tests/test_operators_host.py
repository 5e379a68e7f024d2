"""Host-side checks of the operators of a linear-attention layer: each entry point refuses what it does
not take, with its status and before anything is enqueued.  The pointers are never dereferenced."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import selective_scan_02_b200 as ss
from selective_scan_02_b200._operators import _library

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA, DEVICE = range(7)
FAKE, GB = 0x7F0000000000, 1 << 30


@pytest.fixture(scope="module")
def lib():
    return _library()


def _norm(lib, **kw):
    a = dict(x=FAKE, xd=1, res=None, rd=0, w=FAKE + GB, eps=1e-6, y=FAKE + 2 * GB, yd=1, sc=None, ro=None, rows=4,
             D=256)
    a.update(kw)
    return lib.ss2d_rms_norm(a["x"], a["xd"], a["res"], a["rd"], a["w"], a["eps"], a["y"], a["yd"], a["sc"], a["ro"],
                             a["rows"], a["D"], None)


def test_rms_norm_refusals(lib):
    assert _norm(lib, x=None) == INVALID
    assert _norm(lib, w=None) == INVALID
    assert _norm(lib, y=None) == INVALID
    assert _norm(lib, res=FAKE + 3 * GB) == INVALID and b"together" in lib.ss2d_last_error()
    assert _norm(lib, ro=FAKE + 3 * GB) == INVALID
    assert _norm(lib, yd=2) == INVALID and b"scales" in lib.ss2d_last_error()
    assert _norm(lib, sc=FAKE + 3 * GB) == INVALID
    assert _norm(lib, rows=0) == INVALID
    assert _norm(lib, D=0) == INVALID
    assert _norm(lib, D=32769) == UNSUPPORTED
    assert _norm(lib, eps=-1.0) == INVALID
    assert _norm(lib, eps=float("nan")) == INVALID
    assert _norm(lib, xd=2) == UNSUPPORTED
    assert _norm(lib, xd=3) == UNSUPPORTED
    assert _norm(lib, yd=3) == UNSUPPORTED
    assert _norm(lib, res=FAKE + 3 * GB, ro=FAKE + 4 * GB, rd=2) == UNSUPPORTED
    assert _norm(lib, x=FAKE + 8) == MISALIGNED
    assert _norm(lib, w=FAKE + GB + 4) == MISALIGNED
    assert _norm(lib, y=FAKE) == INVALID and b"overlaps" in lib.ss2d_last_error()
    # the residual in place is one tensor, read and written; a shifted one is not
    shifted = FAKE + 3 * GB
    assert _norm(lib, res=shifted, ro=shifted + 16, rd=1) == INVALID
    assert _norm(lib, res=shifted, ro=FAKE, rd=1) == INVALID
    assert _norm(lib, res=shifted, ro=shifted, rd=1, y=shifted) == INVALID


def _matmul(**kw):
    a = ss.MatmulFp8Args()
    a.struct_size = ctypes.sizeof(a)
    a.M, a.N, a.K = 5, 300, 208
    for i, n in enumerate(("a", "a_scales", "w", "w_scales", "bias", "c")):
        setattr(a, n, FAKE + i * GB)
    a.c_dtype = 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_matmul_fp8_refusals(lib):
    ws = FAKE + 40 * GB
    call = lambda a, w=ws, n=1 << 40: lib.ss2d_matmul_fp8(a, w, n, None)  # noqa: E731
    need = lib.ss2d_matmul_fp8_workspace(_matmul())
    assert 0 < need < 1 << 40
    assert call(_matmul(struct_size=8)) == INVALID
    for name in ("a", "a_scales", "w", "w_scales", "c"):
        assert call(_matmul(**{name: None})) == INVALID
    for name in ("M", "N", "K"):
        assert call(_matmul(**{name: 0})) == INVALID
        assert call(_matmul(**{name: -16})) == INVALID
    assert call(_matmul(K=200)) == UNSUPPORTED and b"16" in lib.ss2d_last_error()
    assert lib.ss2d_matmul_fp8_workspace(_matmul(K=200)) == ctypes.c_size_t(-1).value
    assert call(_matmul(c_dtype=2)) == UNSUPPORTED
    assert call(_matmul(), None) == WORKSPACE
    assert call(_matmul(), ws, need - 1) == WORKSPACE
    assert call(_matmul(), ws + 8) == MISALIGNED
    assert call(_matmul(w=FAKE + 2 * GB + 8)) == MISALIGNED
    assert call(_matmul(c=FAKE)) == INVALID
    assert call(_matmul(), FAKE + 5 * GB) == INVALID  # the workspace overlaps c


def _attention(**kw):
    a = ss.LinearAttentionArgs()
    a.struct_size = ctypes.sizeof(a)
    a.B, a.L, a.G, a.H, a.Dk, a.Dv = 2, 300, 2, 4, 64, 32
    for i, n in enumerate(("q", "k", "v", "log_decay", "h0", "h_last", "out")):
        setattr(a, n, FAKE + i * GB)
    a.q_stride[:] = a.k_stride[:] = (300 * 128, 128, 64)
    a.v_stride[:] = (300 * 128, 128, 32)
    a.scale = 1.0
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def test_linear_attention_refusals(lib):
    ws = FAKE + 40 * GB
    call = lambda a, w=ws, n=1 << 40: lib.ss2d_linear_attention(a, w, n, None)  # noqa: E731
    need = lib.ss2d_linear_attention_workspace(_attention())
    assert 0 < need < 1 << 40
    assert call(_attention(struct_size=8)) == INVALID
    for name in ("q", "k", "v", "log_decay", "out"):
        assert call(_attention(**{name: None})) == INVALID
    for name in ("B", "L", "G", "H", "Dk", "Dv"):
        assert call(_attention(**{name: 0})) == INVALID
    assert call(_attention(H=5)) == INVALID
    assert call(_attention(Dk=136)) == UNSUPPORTED
    assert call(_attention(Dv=136)) == UNSUPPORTED
    assert call(_attention(Dk=60)) == UNSUPPORTED
    assert call(_attention(Dv=4)) == UNSUPPORTED
    assert call(_attention(L=(1 << 24) + 1)) == INVALID
    assert call(_attention(q_stride=(300 * 128, 0, 64))) == UNSUPPORTED   # a broadcast token
    assert call(_attention(q_stride=(300 * 128, 132, 64))) == UNSUPPORTED  # rows off 16 bytes
    assert call(_attention(v_stride=(-8, 128, 32))) == UNSUPPORTED
    assert call(_attention(), None) == WORKSPACE
    assert call(_attention(), ws, need - 1) == WORKSPACE
    assert call(_attention(), ws + 4) == MISALIGNED
    assert call(_attention(q=FAKE + 2)) == MISALIGNED
    assert call(_attention(log_decay=FAKE + 3 * GB + 4)) == MISALIGNED
    assert call(_attention(out=FAKE + 2 * GB)) == INVALID
    assert call(_attention(h_last=FAKE + 4 * GB + 16)) == INVALID  # not in place: it overlaps h0 beside it
    assert call(_attention(), FAKE + 6 * GB) == INVALID


def _step(**kw):
    a = ss.LinearAttentionStepArgs()
    a.struct_size = ctypes.sizeof(a)
    a.B, a.pool, a.G, a.H, a.Dk, a.Dv = 3, 5, 2, 4, 64, 32
    for i, n in enumerate(("q", "k", "v", "log_decay", "slots", "state", "out")):
        setattr(a, n, FAKE + i * GB)
    a.q_stride[:] = a.k_stride[:] = (128, 64)
    a.v_stride[:] = (128, 32)
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def test_linear_attention_step_refusals(lib):
    call = lambda a: lib.ss2d_linear_attention_step(a, None)  # noqa: E731
    assert call(_step(struct_size=8)) == INVALID
    for name in ("q", "k", "v", "log_decay", "state", "out"):
        assert call(_step(**{name: None})) == INVALID
    for name in ("B", "pool", "G", "H", "Dk", "Dv"):
        assert call(_step(**{name: 0})) == INVALID
    assert call(_step(slots=None, pool=2)) == INVALID
    assert call(_step(H=3)) == INVALID
    assert call(_step(Dk=72 * 2)) == UNSUPPORTED
    assert call(_step(k_stride=(128, 4))) == UNSUPPORTED
    assert call(_step(state=FAKE + 5 * GB + 4)) == MISALIGNED
    assert call(_step(out=FAKE + 5 * GB)) == INVALID
    assert call(_step(out=FAKE + 2 * GB)) == INVALID


def test_workspace_status_refusals(lib):
    assert lib.ss2d_workspace_status(None, None) == WORKSPACE
    assert lib.ss2d_workspace_status(FAKE + 4, None) == MISALIGNED


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ss.rms_norm(x, torch.ones(128))
    with pytest.raises(ValueError):
        ss.matmul_fp8(x, x, x, x)
    q = torch.zeros(1, 2, 1, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ss.linear_attention(q, q, q, torch.zeros(1))
    with pytest.raises(ValueError):
        ss.linear_attention_step(q[0], q[0], q[0], torch.zeros(1), torch.zeros(1, 1, 8, 8))


def test_workspace_sizes_refuse_bad_sizes():
    with pytest.raises(ss.Ss2dError):
        ss.matmul_fp8_workspace_size(4, 4, 8)
    with pytest.raises(ss.Ss2dError):
        ss.linear_attention_workspace_size(1, 0, 1, 1, 8, 8)


def test_diag_operator_wait_refusals(lib):
    assert lib.ss2d_diag_operator_wait(None, 1, None) == WORKSPACE
    assert lib.ss2d_diag_operator_wait(FAKE + 4, 1, None) == MISALIGNED
    assert lib.ss2d_diag_operator_wait(FAKE, 0, None) == INVALID
    assert lib.ss2d_diag_operator_wait(FAKE, (1 << 19) + 1, None) == INVALID
    with pytest.raises(ValueError):
        ss.diag_operator_wait(torch.zeros(16, dtype=torch.uint8), 1)


def test_what_is_read_number_by_number_may_lie_on_four_bytes(lib):
    """A refusal that comes behind the alignment's (an overlap of the outputs) shows that the alignment was accepted."""
    ws = FAKE + 40 * GB

    def accepted(status):
        return status == INVALID and b"overlaps" in lib.ss2d_last_error()

    for name in ("a_scales", "w_scales", "bias"):
        at = getattr(_matmul(), name)
        assert accepted(lib.ss2d_matmul_fp8(_matmul(**{name: at + 4, "c": FAKE}), ws, 1 << 40, None)), name
        assert lib.ss2d_matmul_fp8(_matmul(**{name: at + 2, "c": FAKE}), ws, 1 << 40, None) == MISALIGNED
    assert accepted(_norm(lib, yd=2, sc=FAKE + 3 * GB + 4, y=FAKE))
    assert _norm(lib, yd=2, sc=FAKE + 3 * GB + 2, y=FAKE) == MISALIGNED
    assert accepted(lib.ss2d_linear_attention(_attention(lengths=FAKE + 9 * GB + 4, out=FAKE), ws, 1 << 40, None))
    assert lib.ss2d_linear_attention(_attention(lengths=FAKE + 9 * GB + 1, out=FAKE), ws, 1 << 40, None) == MISALIGNED
    assert accepted(lib.ss2d_linear_attention_step(_step(slots=FAKE + 4 * GB + 12, out=FAKE), None))
    assert lib.ss2d_linear_attention_step(_step(slots=FAKE + 4 * GB + 2, out=FAKE), None) == MISALIGNED


def test_no_instance_of_the_norm_that_no_width_takes(lib):
    """The library's own symbols name an instance's threads a row and parts; the entry point's rule names those that it takes,
    for widths that are multiples of 8 and others."""
    names = subprocess.run(["nm", "-C", ss.LIB_PATH], capture_output=True, text=True).stdout
    built = set(re.findall(r"rms_norm_kernel<(\d+), (\d+), (true|false)", names))
    if not built:
        pytest.skip("the library is stripped")
    source = open(os.path.join(os.path.dirname(ss.LIB_PATH), "csrc", "rms_norm.cu")).read()
    rule = set(re.findall(r"e = rms_launch<(\d+), (\d+)>\(a, s\)", source))
    assert {b[:2] for b in built if b[2] == "false"} == {b[:2] for b in built if b[2] == "true"} == rule


def test_a_step_of_too_many_rows_with_slots_is_refused(lib):
    wide = dict(B=65537, pool=65537, H=2, G=2, Dk=8, Dv=8)
    assert lib.ss2d_linear_attention_step(_step(**wide), None) == UNSUPPORTED and b"slots" in lib.ss2d_last_error()
    # without slots it is not (the refusal is the overlap's)
    assert lib.ss2d_linear_attention_step(_step(**wide, slots=None, out=FAKE), None) == INVALID
