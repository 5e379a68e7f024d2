"""Each operator's first call in a process, made inside a graph's capture: nothing that it does once (a kernel's loading, its
shared memory, the tensor maps' encoder) may break the capture."""
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

CODE = """
import sys, torch, selective_scan_02_b200 as ss
which = sys.argv[1]
g = torch.Generator("cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, device="cuda", generator=g)
if which == "norm":
    x, w = r(5, 300).bfloat16(), r(300)
    call = lambda: ss.rms_norm(x, w, residual=x, out_dtype=torch.float8_e4m3fn)
elif which.startswith("matmul"):
    m = int(which[6:])
    a, w = (r(n, 1104).clamp(-4, 4).to(torch.float8_e4m3fn) for n in (m, 520))
    sa, sw = r(m, 9).abs(), r(5, 9).abs()
    call = lambda: (ss.matmul_fp8(a, sa, w, sw),)
else:
    B, L, H = map(int, which.split("x"))
    q, k, v = (r(B, L, h, 64).bfloat16() for h in (1, 1, H))
    gates = torch.full((H,), -0.05, device="cuda")
    if L == 1:
        state = torch.zeros(B, H, 64, 64, device="cuda")
        call = lambda: (ss.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], gates, state.zero_()),)
    else:
        call = lambda: ss.linear_attention(q, k, v, gates, return_last_state=True)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
got = [t.float().clone() for t in out]
want = [t.float() for t in call()]
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
ss.check_workspace_status()
"""


@pytest.mark.parametrize("which", ["norm", "matmul4", "matmul70", "2x1x3", "1x6000x2", "20x700x8"])
def test_first_call_in_a_capture(which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", CODE, which], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
