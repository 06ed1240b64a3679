"""The operators around the scan under sanitizers on the host, and that the checks of their order find
what they are for: in copies of the sources, a barrier and a wait are left out."""

import os
import shutil
import subprocess
import sys

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


def test_bounds(tmp_path):
    r = _run(_build(harness.ROOT, "ops_emu_main.cpp", tmp_path / "asan", "-fsanitize=address", "-fno-omit-frame-pointer"))
    assert r.returncode == 0 and r.stdout.endswith("OK\n"), r.stdout[-500:] + r.stderr[:3000]


def test_no_unordered_access(tmp_path):
    r = _run(_build(harness.ROOT, "ops_emu_main.cpp", tmp_path / "tsan", "-fsanitize=thread"))
    assert "WARNING: ThreadSanitizer" not in r.stderr, r.stderr[:6000]
    assert r.returncode == 0 and r.stdout.endswith("OK\n"), r.stdout[-500:] + r.stderr[-2000:]


def test_a_missing_barrier_is_reported(tmp_path):
    root = _copy(tmp_path, "ssd_gated_kernels.h", "        block_sync();\n        if (SUMMARY) {", "        if (SUMMARY) {")
    r = _run(_build(root, "ops_emu_main.cpp", tmp_path / "planted", "-fsanitize=thread"))
    assert "WARNING: ThreadSanitizer: data race" in r.stderr and "gated_scan_kernel" in r.stderr, r.stderr[-3000:]


@pytest.mark.parametrize("left_out", [False, True])
def test_a_missing_wait_shows(tmp_path, left_out):
    wait = "        async_wait<0>();\n        bare_barrier();"
    root = _copy(tmp_path, "ssd_fp8_kernels.h", wait, wait if not left_out else "        bare_barrier();")
    r = _run(sys.executable, "-c", PLANTED % harness.HERE, _build(root, "ops_emu_lib.cpp", tmp_path / "lib.so", "-fPIC", "-shared"))
    assert ("right" in r.stdout) != left_out, r.stdout + r.stderr[-2000:]
