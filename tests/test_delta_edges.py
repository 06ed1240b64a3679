"""The gated delta rule's further cases (delta_edge_cases) on the CPU, in the host emulator, in one process of its own (this file
run as a program), as test_delta_emulated."""

import os
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import delta_cases as cases
import delta_edge_cases as edges
import delta_emu_harness as harness
from test_delta_boundary import lib  # noqa: F401
from test_delta_emulated import _Run


def everything(lib):
    """(name, function) of every case."""
    run = _Run(lib)
    todo = [("halfway %s" % (c,), lambda c=c: edges.halfway(run, *c)) for c in edges.HALFWAY]
    todo += [("decays %s" % (c,), lambda c=c: edges.decays(run, *c)) for c in edges.DECAYS]
    for c in edges.MANY:
        todo.append(("forward %s" % (c[:7],), lambda c=c: cases.forward(run, *c)))
        todo.append(("backward %s" % (c[:7],), lambda c=c: cases.backward(run, *c)))
    todo += [("outputs %s" % (c[:7],), lambda c=c: edges.outputs(run, *c)) for c in edges.OUTPUTS]
    todo += [("many heads: " + name, fn) for name, fn in edges.many(run)]
    return todo + [("shuffled", lambda: edges.shuffled(run, lib.emu_set_shuffle_seed))]


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    lib = harness.build(str(tmp_path_factory.mktemp("delta_edges")))
    return subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True, text=True)


def test_every_case(report):
    assert report.returncode == 0 and report.stdout.rstrip().endswith("all done"), \
        report.stdout[-2000:] + report.stderr[-2000:]


def test_forms_by_blocks_of_columns(lib):
    """A forward call takes a workspace only where its chunks are packed: the sizes on either side of the bounds where both forms
    were measured."""
    size = lib.ssd_gated_delta_workspace_bytes
    for dtype, Dk, Dv, packed, walked in ((1, 64, 64, 96, 128), (1, 128, 64, 96, 128), (1, 64, 128, 64, 96), (1, 128, 128, 64, 96),
                                          (0, 64, 64, 128, 160), (0, 128, 64, 128, 160), (0, 64, 128, 64, 96), (0, 128, 128, 64, 96)):
        assert size(1, 2048, packed, packed, Dk, Dv, dtype) > 0 and size(1, 2048, walked, walked, Dk, Dv, dtype) == 0


if __name__ == "__main__":
    for name, fn in everything(harness.load(sys.argv[1])):
        print(name, flush=True)
        fn()
    print("all done", flush=True)
