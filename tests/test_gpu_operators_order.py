"""The operators on inputs that change from call to call, written by kernels right ahead of each call on the same stream:
their launches are scheduled before the work ahead is done, and must see what it wrote."""
import pytest
import torch

import selective_scan_02_b200 as ss
from tests.test_gpu_operators import _attention_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _fresh(make, call, rounds=6):
    """call on buffers that are overwritten ahead of every call, against the same call on inputs that have long been there;
    eager and as a replayed graph."""
    sets = [make(i) for i in range(rounds)]
    want = []
    for s in sets:
        torch.cuda.synchronize()
        want.append([t.clone() for t in call(s)])
    bufs = [torch.zeros_like(t) for t in sets[0]]

    def check(run):
        got = []
        for s in sets:
            for b, t in zip(bufs, s):
                b.copy_(t)
            got.append([t.clone() for t in run()])
        for i, (have, w) in enumerate(zip(got, want)):
            assert all(torch.equal(x, y) for x, y in zip(have, w)), i

    check(lambda: call(bufs))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    inputs = [torch.zeros_like(t) for t in sets[0]]
    with torch.cuda.graph(graph):
        for b, t in zip(bufs, inputs):
            b.copy_(t)
        out = call(bufs)

    def replay():
        for b, t in zip(inputs, bufs):
            b.copy_(t)
        graph.replay()
        return out

    check(replay)


# whole heads; segments with a first pass; cut heads; the longest first.  (B, L, G, H, Dk, Dv)
@pytest.mark.parametrize("shape,ragged", [((2, 400, 1, 2, 64, 64), False), ((1, 6000, 1, 2, 128, 96), False),
                                          ((4, 5000, 1, 1, 24, 40), True), ((20, 700, 2, 8, 64, 64), False),
                                          ((40, 650, 1, 4, 16, 24), True), ((30, 500, 1, 10, 128, 32), True),
                                          ((3, 5, 1, 2, 64, 64), True)])
def test_attention_on_fresh_inputs(shape, ragged):
    B, L = shape[:2]

    def make(i):
        q, k, v, gates, _, h0 = _attention_inputs(shape, 300 + i, True, True, False)
        n = torch.randint(0, L + 1, (B,), device="cuda", generator=torch.Generator("cuda").manual_seed(i), dtype=torch.int32)
        return [q, k, v, gates, h0] + ([n] if ragged else [])

    def call(t):
        out = torch.zeros(B, L, shape[3], shape[5], device="cuda", dtype=torch.bfloat16)
        return ss.linear_attention(*t[:4], scale=0.1, h0=t[4], lengths=t[5] if ragged else None, return_last_state=True, out=out)

    _fresh(make, call)


def test_cut_heads_with_a_workspace_of_any_contents():
    """The tickets and marks of cut heads lie in the workspace, whatever it held before."""
    shape = (40, 900, 1, 4, 24, 40)
    q, k, v, gates, scale, h0 = _attention_inputs(shape, 77, True, True, True)
    want = None
    for fill in (0, 1, 127, 128, 255):
        ws = torch.full((ss.linear_attention_workspace_size(*shape),), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            got = ss.linear_attention(q, k, v, gates, scale=scale, h0=h0, return_last_state=True, workspace=ws)
            ss.check_workspace_status(ws)
            want = want or [t.clone() for t in got]
            assert all(torch.equal(a, b) for a, b in zip(got, want))
