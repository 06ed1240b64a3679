"""The operators around the scan: the gated recurrence, the RMS norm, 8-bit
quantisation and the 8-bit product. As for the scan, argument marshalling only (in
the compiled ``_binding.so``): every step runs in the HIP kernels of ``libssd.so`` on
the current stream of the tensors' device, and a call that the library rejects raises
``SSDError``. Tensors of a wrong type, shape, layout or device raise ValueError. Results carry
no autograd history, also of inputs that require gradients: the gradients are calls of their own.

    h, final_state, chunk_states = gated_scan(x, input_gate, decay_gate, lam)
    grads = gated_scan_backward(x, input_gate, decay_gate, lam, chunk_states, grad_h)
    r = rms_norm(x, weight, residual=res, fp8=True)      # r.q, r.scale, r.residual
    grad_x, grad_weight = rms_norm_backward(s, weight, rstd, grad_y)
    q, scale = fp8_quantise(x)                           # 1 x 128 blocks
    y = fp8_matmul(r.q, r.scale, w, w_scale)             # (..., N) bfloat16
"""

from __future__ import annotations

import collections
import ctypes

import torch

GATED_CHUNK = 64  # SSD_GATED_CHUNK
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # SSD_F32, SSD_BF16

GatedScan = collections.namedtuple("GatedScan", "h final_state chunk_states")
GatedGrads = collections.namedtuple("GatedGrads", "x input_gate decay_gate lam initial_state")
RMSNorm = collections.namedtuple("RMSNorm", "y residual q scale rstd")


def declare(lib):
    """Argument types of the operators' entry points."""
    vp, i64, i32, f32, size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                               ctypes.c_size_t)

    def entry(name, res, *args):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = list(args), res

    entry("ssd_gated_scan_workspace_bytes", size, i64, i64, i64, i32)
    entry("ssd_gated_scan", i32, vp, i64, vp, i64, vp, i64, vp, f32, i32, i64, i64, i64, vp, vp, vp,
          vp, vp, vp, size, vp)
    entry("ssd_gated_scan_backward_workspace_bytes", size, i64, i64, i64, i32)
    entry("ssd_gated_scan_backward", i32, vp, i64, vp, i64, vp, i64, vp, f32, i32, i64, i64, i64, vp,
          vp, vp, vp, vp, vp, vp, vp, vp, vp, size, vp)
    entry("ssd_rms_norm", i32, vp, i64, vp, i64, vp, i32, i64, i64, f32, vp, vp, vp, vp, vp, vp)
    entry("ssd_rms_norm_backward_workspace_bytes", size, i64, i64)
    entry("ssd_rms_norm_backward", i32, vp, i64, vp, vp, vp, i64, vp, i64, i32, i64, i64, vp, vp, vp,
          size, vp)
    entry("ssd_fp8_quantise", i32, vp, i64, i32, i64, i64, i64, i32, vp, i64, vp, vp)
    entry("ssd_fp8_matmul_workspace_bytes", size, i64, i64, i64, i64, i32, i32)
    entry("ssd_fp8_matmul", i32, vp, i64, vp, vp, i64, vp, i64, i64, i64, i64, i32, vp, i64, vp, size,
          vp)


_loaded = None


def _binding():
    """The compiled binding (raises OSError if it has not been built)."""
    global _loaded
    if _loaded is None:
        from . import load_library
        lib = load_library()
        try:
            from . import _binding as module
        except ImportError as e:
            raise OSError("_binding.so not loaded (%s); build it with `python -m complex_chunkwise_ssd_amd.build`" % e)
        module.bind(lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
        _loaded = module
    return _loaded


def _size(name, *args) -> int:
    from . import load_library
    return int(getattr(load_library(), name)(*args))


def gated_scan(x, input_gate, decay_gate, lam, decay_scale: float = 8.0, initial_state=None,
               lengths=None, want_final_state: bool = True, want_chunk_states: bool = False, h=None,
               final_state=None, chunk_states=None, workspace=None):
    """The gated linear recurrence, per batch row and channel: with i = sigmoid(input_gate),
    r = sigmoid(decay_gate) and a = exp(-decay_scale softplus(lam) r),
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t.

    x, input_gate, decay_gate (B, T, C) float32 or bfloat16, contiguous or column ranges of
    one (B, T, S) tensor of projected rows; lam (C,) float32; initial_state (B, C) float32;
    lengths (B,) int32: tokens from a row's length on are padding (whatever they hold, h = 0 and
    the state stays). T = 1 is one step of generation; final_state may be initial_state (in place).
    Returns GatedScan(h (B, T, C), final_state (B, C) float32 or None, chunk_states
    (B, ceil(T / 64), C) float32 or None: the states that gated_scan_backward starts from).
    """
    return GatedScan(*(_loaded or _binding()).gated_scan(
        x, input_gate, decay_gate, lam, decay_scale, initial_state, lengths, want_final_state,
        want_chunk_states, h, final_state, chunk_states, workspace))


def gated_scan_backward(x, input_gate, decay_gate, lam, chunk_states, grad_h, grad_final_state=None,
                        decay_scale: float = 8.0, lengths=None, want_initial_state_grad: bool = True,
                        out=None, workspace=None):
    """Gradients of sum(grad_h * h) + sum(grad_final_state * final_state) for the gated_scan
    call with the same inputs; chunk_states as that call returned them. grad_h (B, T, C) in
    x's type, contiguous; grad_final_state (B, C) float32 or None. Returns GatedGrads(x,
    input_gate, decay_gate in x's type (zero in the padding), lam and initial_state float32);
    `out` may supply them."""
    o = out if out is not None else (None, None, None, None, None)
    return GatedGrads(*(_loaded or _binding()).gated_scan_backward(
        x, input_gate, decay_gate, lam, chunk_states, grad_h, grad_final_state, decay_scale, lengths,
        want_initial_state_grad, *o, workspace))


def rms_norm(x, weight, residual=None, eps: float = 1e-6, want_y: bool = True, fp8: bool = False,
             want_rstd: bool = False, y=None, residual_out=None, q=None, scale=None, rstd=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last dimension F.

    x, residual (..., F) float32 or bfloat16 with evenly spaced rows; weight (F,) float32.
    Returns RMSNorm(y in x's type or None, residual = s in x's type (None without a
    residual), q (..., F) float8_e4m3fn and scale (ceil(F / 128), rows) float32 with fp8 (y in 8
    bits, as fp8_matmul reads it), rstd (rows,) float32 if wanted). residual_out may be
    residual (in place)."""
    return RMSNorm(*(_loaded or _binding()).rms_norm(x, weight, residual, eps, want_y, fp8, want_rstd, y,
                                                     residual_out, q, scale, rstd))


def rms_norm_backward(s, weight, rstd, grad_y, grad_residual=None, grad_x=None, grad_weight=None,
                      workspace=None):
    """Gradients of sum(grad_y * y) + sum(grad_residual * s) for rms_norm: s is its residual
    output (its x, where it had no residual), rstd (rows,) as it returned it. Returns
    (grad_x, grad_weight): grad_x (..., F) in s's type is the gradient of x and of residual,
    grad_weight (F,) float32."""
    return (_loaded or _binding()).rms_norm_backward(s, weight, rstd, grad_y, grad_residual, grad_x,
                                                     grad_weight, workspace)


def fp8_quantise(x, block_rows: int = 1, transpose: bool = False, q=None, scale=None):
    """8-bit values (float8_e4m3fn) of x with a float32 scale per block of 128: scale = max |v| /
    448 over the block (at least 2^-126), q = v / scale. x (..., K) float32 or bfloat16 with
    evenly spaced rows, its leading dimensions taken as R rows.

    block_rows 1: 1 x 128 blocks, scale (ceil(K / 128), R); 128: 128 x 128 blocks, scale
    (ceil(R / 128), ceil(K / 128)). With transpose the same of x turned: q (K, R).
    Returns (q, scale). q's rows start on multiples of 16 bytes (K is padded in memory, not in
    shape). fp8_matmul reads such rows as they lie where K is a multiple of 16; for other K its
    form for more than a few rows lays both operands out anew in every call."""
    return (_loaded or _binding()).fp8_quantise(x, block_rows, transpose, q, scale)


def fp8_matmul_workspace_bytes(M, N, K, block_rows=128, out_dtype=torch.bfloat16, rows_on_16=True) -> int:
    return _size("ssd_fp8_matmul_workspace_bytes", M, N, K, block_rows, _DTYPES[out_dtype], rows_on_16)


def gated_scan_workspace_bytes(B, T, C, dtype, backward=False) -> int:
    name = "ssd_gated_scan_backward_workspace_bytes" if backward else "ssd_gated_scan_workspace_bytes"
    return _size(name, B, T, C, _DTYPES[dtype])


def rms_norm_backward_workspace_bytes(rows, F) -> int:
    return _size("ssd_rms_norm_backward_workspace_bytes", rows, F)


def fp8_matmul(a, a_scale, b, b_scale, block_rows: int = 128, out_dtype=torch.bfloat16, out=None,
               workspace=None):
    """out[..., n] = sum over k of (a a_scale)[..., k] (b b_scale)[n, k], both operands 8-bit with a
    scale per block of 128 k. a (..., K) float8_e4m3fn with a_scale (ceil(K / 128), rows) (1 x 128
    blocks); b (N, K) with b_scale (ceil(N / 128), ceil(K / 128)) for block_rows 128, or
    (ceil(K / 128), N) for block_rows 1. Rows evenly spaced. Returns out (..., N) bfloat16 or
    float32; sums are float32."""
    return (_loaded or _binding()).fp8_matmul(a, a_scale, b, b_scale, block_rows, out_dtype, out, workspace)
