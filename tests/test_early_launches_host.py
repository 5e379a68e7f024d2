"""Kernels that are launched before the work ahead of them in their stream is done (launch_early of
selective_scan_02_b200/csrc/launch_util.h) wait for it before they touch global memory, every one and in every thread:
only what stands behind the wait is promised to see what the work ahead wrote."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_scan_02_b200", "csrc")
FILES = [os.path.basename(f) for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "launch_early(" in open(f).read()]


def _source(name):
    """Without comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def _body(src, name):
    """The body of a function, from its definition's opening brace to the closing one."""
    at = re.search(r"\b" + name + r"\s*\((?=[^;{]*\)\s*\{)", src).end()
    start = src.index("{", at)
    depth = 0
    for i in range(start, len(src)):
        depth += (src[i] == "{") - (src[i] == "}")
        if depth == 0:
            return src[start + 1:i]
    raise AssertionError(name)


def _kernels(src):
    return sorted(set(re.findall(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", src)))


def _waits(src, body):
    """Whether a body waits in every thread ahead of any way out: at its outermost level, or in a function that each
    of its branches calls."""
    at = body.find("grid_wait();")
    if at < 0:
        calls = re.findall(r"\b(linear_chunked)<[^;]*?>\(", body)
        return bool(calls) and all(_waits(src, _body(src, c)) for c in calls)
    before = re.sub(r"\[&\]\([^)]*\)\s*\{[^{}]*\}", "", body[:at])  # (without lambdas)
    statement = before[max(before.rfind(";"), before.rfind("}"), before.rfind("{")) + 1:].strip()
    return before.count("{") == before.count("}") and statement == "" and "return" not in before


def test_the_check_itself():
    assert FILES and _waits("", " int a = 1; grid_wait(); x = *p;")
    assert not _waits("", " if (early) grid_wait(); x = *p;")
    assert not _waits("", " if (early) { grid_wait(); } x = *p;")
    assert not _waits("", " if (none) return; grid_wait();")
    assert not _waits("", " x = *p;") and not _waits("", " if (a) { return; } grid_wait();")
    assert _waits("", " auto f = [&](int x) { return x; }; grid_wait();")


@pytest.mark.parametrize("name", FILES)
def test_kernels_wait_for_the_work_ahead(name):
    src = _source(name)
    kernels = _kernels(src)
    assert kernels
    for kernel in kernels:
        assert _waits(src, _body(src, kernel)), kernel


@pytest.mark.parametrize("name", FILES)
def test_nothing_is_read_through_the_read_only_path(name):
    """ld.global.nc may only read what no one writes while the kernel runs; a kernel that is launched early runs while the
    work ahead still writes its inputs."""
    assert not re.search(r"__ldg\b|\.nc\b|__restrict__|__ldlu", _source(name))
