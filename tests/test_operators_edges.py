"""Calls at the edges of what the operators around the scan allow, on the CPU: the unchanged
sources under the host wave emulator, whose buffers end at pages that cannot be touched. Each
case runs in a process of its own (this file run as a program), so that an access past a buffer
ends that process and names its case."""

import os
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import operators_edge_cases as edges
import ops_emu_harness as harness


class _Run:
    """The harness bound to a library."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        return lambda *a, **k: getattr(harness, name)(self._lib, *a, **k)


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    return harness.build(str(tmp_path_factory.mktemp("ops_emu")))


@pytest.mark.parametrize("name", edges.ALL)
def test_edge(library, name):
    r = subprocess.run([sys.executable, os.path.abspath(__file__), library, name], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), "%s: exit status %d\n%s" % (
        name, r.returncode, r.stdout[-1000:] + r.stderr[-2000:])


if __name__ == "__main__":
    edges.ALL[sys.argv[2]](_Run(harness.load(sys.argv[1])))
    print("done")
