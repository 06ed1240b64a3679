"""The gated delta rule with few heads, whose chunks are packed range after range and walked over by a wave for each span
of features: what the form that is taken must not change."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import complex_chunkwise_ssd_amd as ssd
import delta_ref as ref
from test_gpu_delta import _inputs

pytestmark = pytest.mark.gpu


def _part(tensors, at, to):
    return [w[:, at:to].contiguous() for w in tensors]


@pytest.mark.parametrize("sizes,cut", [((2, 9000, 3, 6, 72, 100, "f32"), 4480), ((3, 9000, 4, 16, 40, 64, "f32"), 4480),
                                       ((4, 6000, 3, 12, 128, 48, "bf16"), 2560)])
def test_ranges_of_chunks(sizes, cut):
    """More chunks than are packed at a time: the bits of two calls with the state, or its gradient, handed on
    between them at a chunk's end, and of a call in place."""
    q, k, v, g, beta, init = _inputs(*sizes)
    rows = (q, k, v, g, beta)
    go, gf = torch.randn_like(v.float()).to(v.dtype), torch.randn_like(init)
    whole = ssd.gated_delta(*rows, initial_state=init, want_chunk_states=True)
    first = ssd.gated_delta(*_part(rows, 0, cut), initial_state=init, want_chunk_states=True)
    second = ssd.gated_delta(*_part(rows, cut, None), initial_state=first.final_state, want_chunk_states=True)
    assert torch.equal(whole.o, torch.cat([first.o, second.o], 1))
    assert torch.equal(whole.final_state, second.final_state)
    assert torch.equal(whole.chunk_states, torch.cat([first.chunk_states, second.chunk_states], 1))
    state = init.clone()
    again = ssd.gated_delta(*rows, initial_state=state, final_state=state)
    assert torch.equal(again.o, whole.o) and torch.equal(state, whole.final_state)
    grads = ssd.gated_delta_backward(*rows, whole.chunk_states, go, grad_final_state=gf)
    late = ssd.gated_delta_backward(*_part(rows, cut, None), second.chunk_states, go[:, cut:].contiguous(), grad_final_state=gf)
    early = ssd.gated_delta_backward(*_part(rows, 0, cut), first.chunk_states, go[:, :cut].contiguous(),
                                     grad_final_state=late.initial_state)
    for name in ("q", "k", "v", "g", "beta"):
        assert torch.equal(getattr(grads, name), torch.cat([getattr(early, name), getattr(late, name)], 1)), name
    assert torch.equal(grads.initial_state, early.initial_state)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("Dk", [64, 72, 128])
def test_alone_and_in_a_batch(Dk, kind):
    """The last row's outputs and state have the same bits in a batch of 1, 16 and 64, though the walks have other forms;
    its gradients agree to the order of their sums."""
    B, T, Hv, Dv = 64, 150, 4, 128
    q, k, v, g, beta, init = _inputs(B, T, 2, Hv, Dk, Dv, kind)
    go, gf = torch.randn_like(v.float()).to(v.dtype), torch.randn_like(init)
    got = []
    for n in (1, 16, 64):
        last = [w[B - n:].contiguous() for w in (q, k, v, g, beta, init, go, gf)]
        r = ssd.gated_delta(*last[:5], initial_state=last[5], want_chunk_states=True)
        grads = ssd.gated_delta_backward(*last[:5], r.chunk_states, last[6], grad_final_state=last[7])
        got.append(([w[-1] for w in r], [w[-1].float() for w in grads]))
    for same, near in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(same, got[0][0]))
        for i, (a, b) in enumerate(zip(near, got[0][1])):
            # 64 units of the whole on either side (delta_ref.close), and both results' own rounding
            half = 2 * ref.HALF[kind] if i < 3 else 0.0
            assert (a - b).norm() <= (128 * ref.U + half) * b.norm(), i
