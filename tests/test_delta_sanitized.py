"""The gated delta rule and the norms around a block under sanitizers on the host: reads and writes past a tensor or a
shared-memory array, and accesses of two waves that no barrier orders."""

import os
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import ops_emu_harness as harness
from test_operators_sanitized import _build, _copy, _run


def _bounds(root):
    return _run(_build(harness.ROOT, "delta_emu_main.cpp", root / "asan", "-fsanitize=address", "-fno-omit-frame-pointer"))


def _races(root):
    return _run(_build(harness.ROOT, "delta_emu_main.cpp", root / "tsan", "-fsanitize=thread"))


def _without_barrier(root):
    line = "        block_sync();  // one a chunk: the two halves of what is shared take turns\n        // R"
    copy = _copy(root, "ssd_delta_kernels.h", line, "        // R")
    return _run(_build(copy, "delta_emu_main.cpp", root / "planted", "-fsanitize=thread"))


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    """Every build and run, side by side: name -> its result, once it is there."""
    root = tmp_path_factory.mktemp("delta_sanitized")
    with ThreadPoolExecutor(max_workers=3) as pool:
        futures = {}
        for job in (_bounds, _races, _without_barrier):
            (root / job.__name__).mkdir()
            futures[job.__name__] = pool.submit(job, root / job.__name__)
        yield lambda name: futures[name].result()


def test_bounds(results):
    r = results("_bounds")
    assert r.returncode == 0 and r.stdout.endswith("OK\n"), r.stdout[-500:] + r.stderr[:3000]


def test_no_unordered_access(results):
    r = results("_races")
    assert "WARNING: ThreadSanitizer" not in r.stderr, r.stderr[:6000]
    assert r.returncode == 0 and r.stdout.endswith("OK\n"), r.stdout[-500:] + r.stderr[-2000:]


def test_a_missing_barrier_is_reported(results):
    r = results("_without_barrier")
    assert "WARNING: ThreadSanitizer: data race" in r.stderr and "delta_spans_kernel" in r.stderr, r.stderr[-3000:]
