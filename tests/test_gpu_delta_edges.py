"""The gated delta rule's further cases (delta_edge_cases) on the GPU."""

import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import delta_edge_cases as edges
from test_gpu_delta import _Gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", edges.HALFWAY, ids=str)
def test_halfway(case):
    edges.halfway(_Gpu, *case)
