"""The gated delta rule, and the norms around a block. As in module ops: argument marshalling
only (in the compiled ``_block_binding.so``); every step runs in the HIP kernels of ``libssd.so`` on the
current stream of the tensors' device, a call that the library rejects raises ``SSDError``, and
tensors of a wrong type, shape, layout or device raise ValueError. Results carry no autograd
history: the gradients are calls of their own.

    o, final_state, chunk_states = gated_delta(q, k, v, g, beta)
    grads = gated_delta_backward(q, k, v, g, beta, chunk_states, grad_o)
"""

from __future__ import annotations

import collections
import ctypes

import torch

DELTA_CHUNK = 64  # SSD_DELTA_CHUNK
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # SSD_F32, SSD_BF16

GatedDelta = collections.namedtuple("GatedDelta", "o final_state chunk_states")
DeltaGrads = collections.namedtuple("DeltaGrads", "q k v g beta initial_state")


def declare_delta(lib):
    """Argument types of the delta rule's entry points."""
    vp, i64, i32, f32, size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                               ctypes.c_size_t)

    def entry(name, res, *args):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = list(args), res

    inputs = [vp, i64, vp, i64, vp, i64, vp, vp, f32, i32] + [i64] * 6
    entry("ssd_gated_delta_workspace_bytes", size, *[i64] * 6, i32)
    entry("ssd_gated_delta", i32, *inputs, *[vp] * 6, size, vp)
    entry("ssd_gated_delta_backward_workspace_bytes", size, *[i64] * 6, i32)
    entry("ssd_gated_delta_backward", i32, *inputs, *[vp] * 11, size, vp)


_loaded = None


def _binding():
    """The compiled binding (raises OSError if it has not been built)."""
    global _loaded
    if _loaded is None:
        from . import load_library
        lib = load_library()
        try:
            from . import _block_binding as module
        except ImportError as e:
            raise OSError("_block_binding.so not loaded (%s); build it with `python -m complex_chunkwise_ssd_amd.build`" % e)
        module.bind(lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
        _loaded = module
    return _loaded


def _size(name, *args) -> int:
    from . import load_library
    return int(getattr(load_library(), name)(*args))


def gated_delta(q, k, v, g, beta, scale: float | None = None, initial_state=None, lengths=None,
                want_final_state: bool = True, want_chunk_states: bool = False, o=None,
                final_state=None, chunk_states=None, workspace=None):
    """The gated delta rule, per batch row and value head, on a state S (Dk, Dv): with S' = exp(g_t) S_{t-1}
    and u_t = beta_t (v_t - S'^T k_t), S_t = S' + k_t u_t^T and o_t = scale S_t^T q_t.

    q, k (B, T, Hk, Dk) and v (B, T, Hv, Dv) float32 or bfloat16, contiguous or column ranges of one
    (B, T, S) tensor of projected rows; Hv is a multiple of Hk (neighbouring value heads share a key
    head); Dk <= 128, Dv <= 256. g (log decays, <= 0) and beta (B, T, Hv) float32; scale: Dk^-1/2
    if None. initial_state (B, Hv, Dk, Dv) float32; lengths (B,) int32: tokens from a row's length
    on are padding (whatever they hold, o = 0 and the state stays). Keys are meant to have a
    length of at most 1 (beta |k|^2 in 0 .. 2). T up to 8 is the form for generation;
    final_state may be initial_state (in place).
    Returns GatedDelta(o (B, T, Hv, Dv), final_state (B, Hv, Dk, Dv) float32 or None, chunk_states
    (B, ceil(T / 64), Hv, Dk, Dv) float32 or None: the states that gated_delta_backward starts from).
    """
    return GatedDelta(*(_loaded or _binding()).gated_delta(
        q, k, v, g, beta, scale, initial_state, lengths, want_final_state, want_chunk_states, o, final_state,
        chunk_states, workspace))


def gated_delta_backward(q, k, v, g, beta, chunk_states, grad_o, grad_final_state=None,
                         scale: float | None = None, lengths=None, want_initial_state_grad: bool = True,
                         out=None, workspace=None):
    """Gradients of sum(grad_o * o) + sum(grad_final_state * final_state) for the gated_delta call with
    the same inputs; chunk_states as that call returned them. grad_o (B, T, Hv, Dv) in v's
    type, contiguous; grad_final_state (B, Hv, Dk, Dv) float32 or None. Returns DeltaGrads(q, k, v in
    their type (q and k summed over the value heads that share a key head), g and beta (B, T, Hv)
    and initial_state float32), zero in the padding; `out` may supply them."""
    args = out if out is not None else (None,) * 6
    return DeltaGrads(*(_loaded or _binding()).gated_delta_backward(
        q, k, v, g, beta, chunk_states, grad_o, grad_final_state, scale, lengths, want_initial_state_grad, *args,
        workspace))


def gated_delta_workspace_bytes(B, T, Hk, Hv, Dk, Dv, dtype, backward=False) -> int:
    name = "ssd_gated_delta_backward_workspace_bytes" if backward else "ssd_gated_delta_workspace_bytes"
    return _size(name, B, T, Hk, Hv, Dk, Dv, _DTYPES[dtype])
