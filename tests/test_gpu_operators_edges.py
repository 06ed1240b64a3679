"""Calls at the edges of what the operators around the scan allow, on the GPU through the Python
entry points: the emulator's cases."""

import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import operators_edge_cases as edges
from test_gpu_operators import _Gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", edges.ALL)
def test_edge(name):
    edges.ALL[name](_Gpu)
