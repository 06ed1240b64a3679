"""Which library the compiled binding of the operators calls, on the CPU."""

import os
import shutil
import subprocess
import sys

import pytest

import complex_chunkwise_ssd_amd as ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import ctypes, sys
import complex_chunkwise_ssd_amd as ssd
other = ssd.load_library(sys.argv[1])
binding = ssd.ops._binding()
mine = ssd.load_library()
at = lambda lib, name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
print("bound", all(a == at(mine, n) != at(other, n) for n, a in binding.bound().items()), len(binding.bound()))
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(ssd.LIBPATH):
        from complex_chunkwise_ssd_amd import build
        build.build()


def test_the_binding_calls_the_library_of_the_package(tmp_path):
    """Another copy of the library that the process loaded before does not take its place."""
    other = str(tmp_path / "libssd.so")
    shutil.copy(ssd.LIBPATH, other)
    r = subprocess.run([sys.executable, "-c", PROGRAM, other], cwd=ROOT, capture_output=True, text=True,
                       env={**os.environ, "LD_DEBUG": "bindings", "LD_BIND_NOW": "1"})
    to_other = [line for line in r.stderr.splitlines() if "_binding.so" in line and "to %s" % other in line]
    assert not to_other, to_other[:3]
    assert r.returncode == 0 and "bound True 10" in r.stdout, r.stdout + r.stderr[-2000:]
