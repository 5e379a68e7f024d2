"""The operators' bounded waits, run out on purpose: reported by the workspace and by the device, by a context that stays
usable.  No fault, trap or hang is involved: every wait ends."""
import pytest
import torch

import selective_scan_02_b200 as ss
from tests.test_gpu_operators import _attention_inputs, _check_attention, _check_matmul, _matmul_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_a_wait_that_runs_out_is_reported():
    ss.check_workspace_status()
    a, sa, w, sw, _ = _matmul_inputs(40, 200, 256, 71)
    shape = (1, 300, 1, 2, 64, 64)
    q, k, v, gates, scale, h0 = _attention_inputs(shape, 72, True, True, False)
    ws = torch.full((max(ss.matmul_fp8_workspace_size(40, 200, 256), ss.linear_attention_workspace_size(*shape)),), 255,
                    dtype=torch.uint8, device="cuda")
    for limit in (1, 2048):
        ss.diag_operator_wait(ws, limit)
        for check in (lambda: ss.check_workspace_status(ws), ss.check_workspace_status):
            with pytest.raises(ss.Ss2dError) as e:
                check()
            assert e.value.name == "SS2D_ERR_DEVICE"
        ss.check_workspace_status()  # it has been said
    # the next calls clear the workspace's word, run and are right
    got = ss.matmul_fp8(a, sa, w, sw, workspace=ws)
    ss.check_workspace_status(ws)
    _check_matmul(got, a, sa, w, sw, None)
    ss.diag_operator_wait(ws, 1)
    out, last = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True, workspace=ws)
    ss.check_workspace_status(ws)
    _check_attention(q, k, v, gates, scale, h0, None, out, last)
    # what the workspace no longer says, the device does, on whatever stream it is asked
    with pytest.raises(ss.Ss2dError):
        ss.check_workspace_status(stream=torch.cuda.Stream())
    ss.check_workspace_status()


def test_calls_without_a_workspace_can_be_asked_about():
    a, sa, w, sw, _ = _matmul_inputs(4, 64, 128, 73)
    ss.matmul_fp8(a, sa, w, sw)
    ss.check_workspace_status()
    ss.check_workspace_status(stream=torch.cuda.current_stream())


def test_refusals():
    with pytest.raises(ValueError):
        ss.check_workspace_status(torch.zeros(16, 16, device="cuda").t()[:, :3])
    with pytest.raises(ValueError):
        ss.check_workspace_status(torch.zeros(2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ss.diag_operator_wait(torch.zeros(2, dtype=torch.uint8, device="cuda"), 1)
    for limit in (0, (1 << 19) + 1):
        with pytest.raises(ss.Ss2dError):
            ss.diag_operator_wait(torch.zeros(16, dtype=torch.uint8, device="cuda"), limit)
