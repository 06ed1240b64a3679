"""The gated delta rule's further cases (delta_edge_cases) on the GPU."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import complex_chunkwise_ssd_amd as ssd
import delta_cases as cases
import delta_edge_cases as edges
from test_gpu_delta import _both, _Gpu, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", edges.HALFWAY, ids=str)
def test_halfway(case):
    edges.halfway(_Gpu, *case)


@pytest.mark.parametrize("case", edges.DECAYS, ids=str)
def test_decays(case):
    edges.decays(_Gpu, *case)


@pytest.mark.parametrize("case", edges.MANY, ids=lambda c: str(c[:7]))
def test_many_heads(case):
    cases.forward(_Gpu, *case)


@pytest.mark.parametrize("case", edges.MANY, ids=lambda c: str(c[:7]))
def test_many_heads_backward(case):
    cases.backward(_Gpu, *case)


@pytest.mark.parametrize("case", edges.OUTPUTS, ids=lambda c: str(c[:7]))
def test_outputs(case):
    edges.outputs(_Gpu, *case)


@pytest.mark.parametrize("name,fn", edges.many(_Gpu), ids=lambda x: x if isinstance(x, str) else "")
def test_many_heads_as_few(name, fn):
    fn()


def _off(t):
    """The same values one element past a boundary."""
    wide = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    wide[1:] = t.reshape(-1)
    return wide[1:].view(t.shape)


@pytest.mark.parametrize("sizes", [(2, 140, 1, 2, 32, 40, "f32"), (2, 140, 1, 1, 72, 68, "bf16"), (97, 140, 1, 2, 64, 64, "bf16"),
                                   (97, 70, 2, 2, 72, 36, "f32"), (97, 70, 1, 1, 128, 128, "bf16"), (3, 4, 1, 2, 24, 20, "bf16")])
def test_tensors_one_element_off(sizes):
    """Alignment to the element is all that is asked for: the same bits."""
    *args, init = _inputs(*sizes)
    want = _both(args, init, args[2])
    got = _both([_off(w) for w in args], _off(init), _off(args[2]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    states = want[2]
    grads = ssd.gated_delta_backward(*args, _off(states), args[2], grad_final_state=init)
    assert all(torch.equal(a, b) for a, b in zip(grads, want[3:]))


@pytest.mark.parametrize("B,T", [(1, 140000), (700, 200), (30000, 5)])
def test_rows_whose_offsets_pass_32_bits(B, T):
    """q, k and v as column ranges of 2.3e9 elements, in a sequence, in a batch and token by token: the bits of dense ones."""
    *args, init = _inputs(B, T, 1, 2, 64, 32, "bf16")
    rows = torch.full((B, T, 1 << 14), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    parts, at = [], (1 << 14) - 192
    for w in args[:3]:
        n = w[0, 0].numel()
        rows[..., at:at + n] = w.flatten(2)
        parts.append(rows[..., at:at + n].unflatten(-1, w.shape[2:]))
        at += n
    want = _both(args, init, args[2])
    got = _both([*parts, *args[3:]], init, args[2])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_workspace_one_call_after_another():
    """Calls of several sizes and directions share one workspace on a stream; what it held does not matter."""
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda:0")
    for sizes in ((2, 300, 2, 4, 64, 64, "bf16"), (97, 130, 1, 2, 72, 48, "f32"), (3, 130, 1, 2, 100, 40, "f32"), (2, 5, 1, 2, 64, 64, "bf16")):
        *args, init = _inputs(*sizes)
        want = _both(args, init, args[2])
        for _ in range(2):
            r = ssd.gated_delta(*args, initial_state=init, want_chunk_states=True, workspace=ws)
            grads = ssd.gated_delta_backward(*args, r.chunk_states, args[2], grad_final_state=init, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip([*r, *grads], want))
