"""The operators around the scan under sanitizers on the host, and that the checks of their order find
what they are for: in copies of the sources, a barrier and a wait are left out."""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import ops_emu_harness as harness

PLANTED = """
import sys
sys.path.insert(0, %r)
import operators_cases as cases, ops_emu_harness as harness
from test_operators_edges import _Run
cases.matmul(_Run(harness.load(sys.argv[1])), 70, 90, 400, 128, "bf16", 0, 0, 0)
print("right")
"""


def _build(source_root, main, out, *flags):
    emu = os.path.join(source_root, "tests", "emu")
    subprocess.run([harness.CLANG, "-x", "c++", "-std=c++17", "-I" + emu,
                    "-I" + os.path.join(source_root, "complex_chunkwise_ssd_amd", "csrc"),
                    "-I" + os.path.join(harness.ROOT, "include"), "-O1", "-g", "-Wno-psabi", *flags,
                    os.path.join(emu, main), "-o", str(out)], check=True)
    return str(out)


def _copy(root, header, old, new):
    """The sources with one place changed."""
    shutil.copytree(harness.EMU, root / "tests" / "emu")
    shutil.copytree(harness.CSRC, root / "complex_chunkwise_ssd_amd" / "csrc")
    path = root / "complex_chunkwise_ssd_amd" / "csrc" / header
    text = path.read_text()
    assert text.count(old) == 1
    path.write_text(text.replace(old, new))
    return str(root)


def _run(*cmd):
    return subprocess.run(cmd, capture_output=True, text=True, timeout=600,
                          env={**os.environ, "TSAN_OPTIONS": "halt_on_error=1"})


def _bounds(root):
    return _run(_build(harness.ROOT, "ops_emu_main.cpp", root / "asan", "-fsanitize=address", "-fno-omit-frame-pointer"))


def _races(root):
    return _run(_build(harness.ROOT, "ops_emu_main.cpp", root / "tsan", "-fsanitize=thread"))


def _without_barrier(root):
    copy = _copy(root, "ssd_gated_kernels.h", "        block_sync();\n        if (SUMMARY) {", "        if (SUMMARY) {")
    return _run(_build(copy, "ops_emu_main.cpp", root / "planted", "-fsanitize=thread"))


WAIT = "        async_wait<0>();\n        bare_barrier();"


def _with_wait(root, wait=WAIT):
    copy = _copy(root, "ssd_fp8_kernels.h", WAIT, wait)
    return _run(sys.executable, "-c", PLANTED % harness.HERE, _build(copy, "ops_emu_lib.cpp", root / "lib.so", "-fPIC", "-shared"))


def _without_wait(root):
    return _with_wait(root, "        bare_barrier();")


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    """Every build and run, side by side: name -> its result, once it is there."""
    root = tmp_path_factory.mktemp("sanitized")
    with ThreadPoolExecutor(max_workers=5) as pool:
        futures = {}
        for job in (_bounds, _races, _without_barrier, _with_wait, _without_wait):
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
    assert "WARNING: ThreadSanitizer: data race" in r.stderr and "gated_scan_kernel" in r.stderr, r.stderr[-3000:]


def test_a_missing_wait_shows(results):
    r = results("_with_wait")
    assert r.returncode == 0 and "right" in r.stdout, r.stdout + r.stderr[-2000:]
    r = results("_without_wait")
    assert r.returncode != 0 and "right" not in r.stdout and ("off, worst" in r.stderr or "emu:" in r.stderr), \
        r.stdout + r.stderr[-2000:]
