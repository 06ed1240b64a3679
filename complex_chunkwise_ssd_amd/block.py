"""The gated delta rule, and the norms around a block. As in module ops: argument marshalling
only (in the compiled ``_block_binding.so``); every step runs in the HIP kernels of ``libssd.so`` on the
current stream of the tensors' device, a call that the library rejects raises ``SSDError``, and
tensors of a wrong type, shape, layout or device raise ValueError. Results carry no autograd
history: the gradients are calls of their own.

    o, final_state, chunk_states = gated_delta(q, k, v, g, beta)
    grads = gated_delta_backward(q, k, v, g, beta, chunk_states, grad_o)
    n = gated_norm(o.flatten(-2), z, weight, fp8=True)                 # n.q, n.scale
    b = block_norm(x, residual, post_weight, pre_weight, fp8=True)     # b.q, b.scale, b.residual
"""

from __future__ import annotations

import collections
import ctypes

import torch

DELTA_CHUNK = 64  # SSD_DELTA_CHUNK
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # SSD_F32, SSD_BF16

GatedDelta = collections.namedtuple("GatedDelta", "o final_state chunk_states")
DeltaGrads = collections.namedtuple("DeltaGrads", "q k v g beta initial_state")
GatedNorm = collections.namedtuple("GatedNorm", "y q scale rstd")
GatedNormGrads = collections.namedtuple("GatedNormGrads", "x gate weight")
BlockNorm = collections.namedtuple("BlockNorm", "y residual q scale post_rstd pre_rstd")
BlockNormGrads = collections.namedtuple("BlockNormGrads", "x residual post_weight pre_weight")


_VP, _I64, _I32, _F32, _SIZE = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                ctypes.c_size_t)


def _entry(lib, name, res, *args):
    fn = getattr(lib, name)
    fn.argtypes, fn.restype = list(args), res


def declare_delta(lib):
    """Argument types of the delta rule's entry points."""
    vp, i64, i32, f32, size = _VP, _I64, _I32, _F32, _SIZE
    inputs = [vp, i64, vp, i64, vp, i64, vp, vp, f32, i32] + [i64] * 6
    _entry(lib, "ssd_gated_delta_workspace_bytes", size, *[i64] * 6, i32)
    _entry(lib, "ssd_gated_delta", i32, *inputs, *[vp] * 6, size, vp)
    _entry(lib, "ssd_gated_delta_backward_workspace_bytes", size, *[i64] * 6, i32)
    _entry(lib, "ssd_gated_delta_backward", i32, *inputs, *[vp] * 11, size, vp)


def declare_norms(lib):
    """Argument types of the norms' entry points."""
    vp, i64, i32, f32, size = _VP, _I64, _I32, _F32, _SIZE
    _entry(lib, "ssd_gated_norm", i32, vp, i64, vp, i64, vp, i32, i64, i64, i64, f32, vp, vp, vp, vp, vp)
    _entry(lib, "ssd_gated_norm_backward_workspace_bytes", size, i64, i64, i64)
    _entry(lib, "ssd_gated_norm_backward", i32, vp, i64, vp, i64, vp, vp, vp, i64, i32, i64, i64, i64, vp, vp, vp,
           vp, size, vp)
    _entry(lib, "ssd_block_norm", i32, vp, i64, vp, i64, vp, vp, f32, i32, i64, i64, f32, *[vp] * 6, vp)
    _entry(lib, "ssd_block_norm_backward_workspace_bytes", size, i64, i64)
    _entry(lib, "ssd_block_norm_backward", i32, vp, i64, vp, i64, vp, vp, vp, vp, f32, vp, i64, vp, i64, i32, i64, i64,
           vp, vp, vp, vp, vp, size, vp)


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
    (B, T, S) tensor of projected rows (a range of tokens of several rows has to be copied first); Hv is a multiple of Hk (neighbouring value heads share a key
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


def gated_norm(x, gate, weight, eps: float = 1e-6, want_y: bool = True, fp8: bool = False, want_rstd: bool = False,
               y=None, q=None, scale=None, rstd=None):
    """The norm of a mixer's outputs by heads, fused with their gate: y = x / sqrt(mean(x^2) + eps) * weight *
    silu(gate), the mean over each D neighbours of the last dimension F.

    x, gate (..., F) float32 or bfloat16 with evenly spaced rows; weight (D,) float32, D >= 8 a divisor of F
    (the same weights for every head). Returns GatedNorm(y in x's type or None, q (..., F)
    float8_e4m3fn and scale (ceil(F / 128), rows) float32 with fp8 (y in 8 bits, as fp8_matmul reads
    it), rstd (rows, F / D) float32 if wanted)."""
    return GatedNorm(*(_loaded or _binding()).gated_norm(x, gate, weight, eps, want_y, fp8, want_rstd, y, q, scale,
                                                         rstd))


def gated_norm_backward(x, gate, weight, rstd, grad_y, grad_x=None, grad_gate=None, grad_weight=None, workspace=None):
    """Gradients of sum(grad_y * y) for gated_norm; rstd (rows, F / D) as it returned it. Returns
    GatedNormGrads(x, gate (..., F) in x's type, weight (D,) float32, summed over rows and heads)."""
    return GatedNormGrads(*(_loaded or _binding()).gated_norm_backward(x, gate, weight, rstd, grad_y, grad_x, grad_gate,
                                                                       grad_weight, workspace))


def gated_norm_backward_workspace_bytes(rows, F, D) -> int:
    return _size("ssd_gated_norm_backward_workspace_bytes", rows, F, D)


def block_norm(x, residual, post_weight, pre_weight, residual_scale: float = 1.0, eps: float = 1e-6,
               want_y: bool = True, fp8: bool = False, want_rstd: bool = False, y=None, residual_out=None, q=None,
               scale=None, post_rstd=None, pre_rstd=None):
    """The end of a block and the start of the next: s = residual + residual_scale * x / sqrt(mean(x^2) + eps) *
    post_weight, y = s / sqrt(mean(s^2) + eps) * pre_weight, over the last dimension F.

    x, residual (..., F) float32 or bfloat16 with evenly spaced rows; both weights (F,) float32. Returns
    BlockNorm(y in x's type or None, residual = s in x's type, q (..., F) float8_e4m3fn and scale
    (ceil(F / 128), rows) float32 with fp8 (y in 8 bits, as fp8_matmul reads it), post_rstd and pre_rstd
    (rows,) float32 if wanted). residual_out may be residual (in place)."""
    return BlockNorm(*(_loaded or _binding()).block_norm(x, residual, post_weight, pre_weight, residual_scale, eps,
                                                         want_y, fp8, want_rstd, y, residual_out, q, scale, post_rstd,
                                                         pre_rstd))


def block_norm_backward(x, s, post_weight, pre_weight, post_rstd, pre_rstd, grad_y, grad_residual=None,
                        residual_scale: float = 1.0, grad_x=None, grad_residual_in=None, grad_post_weight=None,
                        grad_pre_weight=None, workspace=None):
    """Gradients of sum(grad_y * y) + sum(grad_residual * s) for block_norm: s is its residual output, the rstds
    (rows,) as it returned them. Returns BlockNormGrads(x, residual (..., F) in x's type, post_weight,
    pre_weight (F,) float32)."""
    return BlockNormGrads(*(_loaded or _binding()).block_norm_backward(
        x, s, post_weight, pre_weight, post_rstd, pre_rstd, grad_y, grad_residual, residual_scale, grad_x,
        grad_residual_in, grad_post_weight, grad_pre_weight, workspace))


def block_norm_backward_workspace_bytes(rows, F) -> int:
    return _size("ssd_block_norm_backward_workspace_bytes", rows, F)
