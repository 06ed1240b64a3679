"""The gated delta rule on the host with every access held to the alignment that its type promises (a load by vectors of four
floats may be compiled into one that needs 16 bytes), and with signed sums and products held to their range."""

import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import ops_emu_harness as harness
from test_operators_sanitized import _build, _run


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return _build(harness.ROOT, "delta_align_main.cpp", tmp_path_factory.mktemp("delta_alignment") / "align",
                  "-fsanitize=alignment,signed-integer-overflow", "-fno-sanitize-recover=all")


def test_tensors_on_a_boundary(program):
    r = _run(program, "0")
    assert r.returncode == 0 and "\nOK " in r.stdout, r.stdout[-500:] + r.stderr[:3000]


def test_tensors_one_element_off(program):
    """Alignment to the element is all that the header asks for: the same results, bit for bit."""
    r = _run(program, "1")
    assert r.returncode == 0 and "\nOK " in r.stdout, r.stdout[-500:] + r.stderr[:3000]
    assert r.stdout == _run(program, "0").stdout


def test_sizes_past_the_limits(program):
    r = _run(program, "limits")
    assert r.returncode == 0 and r.stdout == "OK \n", r.stdout + r.stderr[:3000]
