"""The operators' calls and Python's other threads: a call that waits, for its stream or for room in the queue of launches,
holds none of them up."""
import threading
import time

import pytest
import torch

import selective_scan_02_b200 as ss

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class _Ticks:
    """A thread that notes the time about every millisecond."""

    def __enter__(self):
        self.at, self.stop = [time.perf_counter()], False
        self.thread = threading.Thread(target=self._run)
        self.thread.start()
        return self

    def _run(self):
        while not self.stop:
            time.sleep(0.001)
            self.at.append(time.perf_counter())

    def __exit__(self, *_):
        self.stop = True
        self.thread.join()

    def widest(self, start, end):
        at = [start] + [t for t in self.at if start < t < end] + [end]
        return max(b - a for a, b in zip(at, at[1:]))


def _busy(seconds):
    """Work for the GPU that lasts about so long, enqueued in a few launches."""
    a = torch.randn(8192, 8192, device="cuda").bfloat16()
    out = torch.empty_like(a)
    torch.mm(a, a, out=out)
    torch.cuda.synchronize()
    start = time.perf_counter()
    torch.mm(a, a, out=out)
    torch.cuda.synchronize()
    each = time.perf_counter() - start
    return lambda: [torch.mm(a, a, out=out) for _ in range(int(seconds / each) + 1)]


def test_a_status_that_waits():
    ws = torch.zeros(ss.matmul_fp8_workspace_size(4, 64, 128), dtype=torch.uint8, device="cuda")
    busy = _busy(0.3)
    with _Ticks() as ticks:
        busy()
        start = time.perf_counter()
        ss.check_workspace_status(ws)
        end = time.perf_counter()
    assert end - start > 0.1, "the GPU was not busy"
    assert ticks.widest(start, end) < (end - start) / 2


def test_launches_that_wait_for_room():
    x = torch.randn(4, 256, device="cuda").bfloat16()
    w, y = torch.ones(256, device="cuda"), torch.empty_like(x)
    ss.rms_norm(x, w, y=y)
    torch.cuda.synchronize()
    busy = _busy(0.4)
    with _Ticks() as ticks:
        busy()
        start = time.perf_counter()
        for _ in range(6000):  # more than the queue holds
            ss.rms_norm(x, w, y=y)
        end = time.perf_counter()
        torch.cuda.synchronize()
    assert end - start > 0.1, "no launch waited"
    assert ticks.widest(start, end) < (end - start) / 2


def test_calls_from_several_threads():
    """Threads that call at once, each on a stream of its own; the first of them makes the first calls of its kinds."""
    g = torch.Generator("cuda").manual_seed(5)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=g)

    def attention(B, L, H, D):
        q, v, gates = normal(B, L, 1, D).bfloat16(), normal(B, L, H, D).bfloat16(), torch.full((H,), -0.03, device="cuda")
        return lambda: ss.linear_attention(q, q, v, gates, return_last_state=True)

    def product(m, n, k):
        a, w = (normal(x, k).clamp(-4, 4).to(torch.float8_e4m3fn) for x in (m, n))
        sa, sw = normal(m, -(-k // 128)).abs(), normal(-(-n // 128), -(-k // 128)).abs()
        return lambda: (ss.matmul_fp8(a, sa, w, sw),)

    def norm(rows, d):
        x, w = normal(rows, d), normal(d)
        return lambda: ss.rms_norm(x, w, out_dtype=torch.float8_e4m3fn)

    calls = [attention(20, 700, 8, 64), attention(1, 6000, 2, 96), attention(3, 6, 2, 40), product(5, 300, 1104),
             product(90, 300, 2048), norm(40, 1000)]
    got = [[] for _ in calls]
    failed = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i].append(calls[i]())
                s.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for call, results in zip(calls, got):
        want = call()
        assert len(results) == 20 and all(torch.equal(x.float(), y.float()) for r in results for x, y in zip(r, want))
    ss.check_workspace_status()
