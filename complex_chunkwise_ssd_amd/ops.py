"""The operators around the scan: the gated recurrence, the RMS norm, 8-bit
quantisation and the 8-bit product. As for the scan, argument marshalling only:
every step runs in the HIP kernels of ``libssd.so`` on the current stream of the
tensors' device, and a call that the library rejects raises ``SSDError``.

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


_entries = {}  # name -> function of the loaded library


def _entry(name):
    fn = _entries.get(name)
    if fn is None:
        from . import load_library
        fn = _entries[name] = getattr(load_library(), name)
    return fn


# The stream as an integer; the public way builds a Stream object first (1.5 us of a 10 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """One entry point on the current stream of `dev`, which becomes the current device for
    the call if it is not."""
    fn = _entries.get(name) or _entry(name)
    index = dev.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        from . import SSDError
        raise SSDError(st, name)


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device, got %s" % dev)
    return dev


def _dtype(t, name):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return dt


def _check(t, name, dtype, shape, dev):
    """A dense tensor of this type, shape and device."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _out(t, name, dtype, shape, dev, want=True):
    """The output that was passed in, checked, or a new one (None if it is not wanted)."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if want else None
    _check(t, name, dtype, shape, dev)
    return t


def _workspace(ws, n, dev):
    if ws is None:
        return (torch.empty(n, dtype=torch.uint8, device=dev), n) if n else (None, 0)
    if not isinstance(ws, torch.Tensor) or ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    return ws, ws.numel() * ws.element_size()


def _row_stride(t, name, dtype, shape, dev):
    """Elements between the rows of t (..., F): its last dimension dense, the rows evenly
    spaced (a contiguous tensor, or a column range of one)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype or t.device != dev or t.shape != shape:
        raise ValueError("%s must be %s of shape %s on %s, got %s of shape %s on %s" % (
            name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape), t.device))
    F = shape[-1]
    if t.is_contiguous():
        return F
    strides = t.stride()
    want = step = None  # between neighbouring rows; that the next dimension out has to have
    for d in range(len(shape) - 2, -1, -1):
        if shape[d] == 1:
            continue
        if want is None:
            want = step = strides[d]
        if strides[d] != step:
            want = 0
            break
        step *= shape[d]
    if F > 1 and strides[-1] != 1:
        want = 0
    if want is None:
        want = F
    if want < F:
        raise ValueError("%s must have a dense last dimension and evenly spaced rows, got strides %s"
                         % (name, strides))
    return want


def _rows(shape):
    n = 1
    for d in shape:
        n *= int(d)
    return n


def _gated_inputs(x, input_gate, decay_gate, lam, lengths):
    dev = _device(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be a (B, T, C) tensor")
    dt = _dtype(x, "x")
    B, T, C = x.shape
    shape, ty = x.shape, x.dtype
    strides = (_row_stride(x, "x", ty, shape, dev),
               _row_stride(input_gate, "input_gate", ty, shape, dev),
               _row_stride(decay_gate, "decay_gate", ty, shape, dev))
    _check(lam, "lam", torch.float32, (C,), dev)
    if lengths is not None:
        _check(lengths, "lengths", torch.int32, (B,), dev)
    return dev, dt, B, T, C, strides


def gated_scan(x, input_gate, decay_gate, lam, decay_scale: float = 8.0, initial_state=None,
               lengths=None, want_final_state: bool = True, want_chunk_states: bool = False, h=None,
               final_state=None, chunk_states=None, workspace=None):
    """The gated linear recurrence, per batch row and channel: with i = sigmoid(input_gate),
    r = sigmoid(decay_gate) and a = exp(-decay_scale softplus(lam) r),
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t.

    x, input_gate, decay_gate (B, T, C) float32 or bfloat16, contiguous or column ranges of
    one (B, T, S) tensor of projected rows; lam (C,) float32; initial_state (B, C) float32;
    lengths (B,) int32: tokens from a row's length on are padding (not read, h = 0, the state
    stays). T = 1 is one step of generation; final_state may be initial_state (in place).
    Returns GatedScan(h (B, T, C), final_state (B, C) float32 or None, chunk_states
    (B, ceil(T / 64), C) float32 or None: the states that gated_scan_backward starts from).
    """
    dev, dt, B, T, C, st = _gated_inputs(x, input_gate, decay_gate, lam, lengths)
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (B, C), dev)
    h = _out(h, "h", x.dtype, (B, T, C), dev)
    final_state = _out(final_state, "final_state", torch.float32, (B, C), dev, want_final_state)
    chunk_states = _out(chunk_states, "chunk_states", torch.float32,
                        (B, -(-T // GATED_CHUNK), C), dev, want_chunk_states)
    ws, size = _workspace(workspace, _entry("ssd_gated_scan_workspace_bytes")(B, T, C, dt), dev)
    _call("ssd_gated_scan", dev, _ptr(x), st[0], _ptr(input_gate), st[1], _ptr(decay_gate), st[2],
          _ptr(lam), float(decay_scale), dt, B, T, C, _ptr(initial_state), _ptr(lengths), _ptr(h),
          _ptr(final_state), _ptr(chunk_states), _ptr(ws), size)
    return GatedScan(h, final_state, chunk_states)


def gated_scan_backward(x, input_gate, decay_gate, lam, chunk_states, grad_h, grad_final_state=None,
                        decay_scale: float = 8.0, lengths=None, want_initial_state_grad: bool = True,
                        out=None, workspace=None):
    """Gradients of sum(grad_h * h) + sum(grad_final_state * final_state) for the gated_scan
    call with the same inputs; chunk_states as that call returned them. grad_h (B, T, C) in
    x's type, contiguous; grad_final_state (B, C) float32 or None. Returns GatedGrads(x,
    input_gate, decay_gate in x's type (zero in the padding), lam and initial_state float32);
    `out` may supply them."""
    dev, dt, B, T, C, st = _gated_inputs(x, input_gate, decay_gate, lam, lengths)
    _check(chunk_states, "chunk_states", torch.float32, (B, -(-T // GATED_CHUNK), C), dev)
    _check(grad_h, "grad_h", x.dtype, (B, T, C), dev)
    if grad_final_state is not None:
        _check(grad_final_state, "grad_final_state", torch.float32, (B, C), dev)
    o = out if out is not None else GatedGrads(None, None, None, None, None)
    gx, gi, gr = (_out(t, n, x.dtype, (B, T, C), dev) for t, n in (
        (o.x, "grad x"), (o.input_gate, "grad input_gate"), (o.decay_gate, "grad decay_gate")))
    glam = _out(o.lam, "grad lam", torch.float32, (C,), dev)
    ginit = _out(o.initial_state, "grad initial_state", torch.float32, (B, C), dev,
                 want_initial_state_grad)
    ws, size = _workspace(workspace, _entry("ssd_gated_scan_backward_workspace_bytes")(B, T, C, dt), dev)
    _call("ssd_gated_scan_backward", dev, _ptr(x), st[0], _ptr(input_gate), st[1], _ptr(decay_gate),
          st[2], _ptr(lam), float(decay_scale), dt, B, T, C, _ptr(chunk_states), _ptr(lengths),
          _ptr(grad_h), _ptr(grad_final_state), _ptr(gx), _ptr(gi), _ptr(gr), _ptr(glam),
          _ptr(ginit), _ptr(ws), size)
    return GatedGrads(gx, gi, gr, glam, ginit)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, want_y: bool = True, fp8: bool = False,
             want_rstd: bool = False, y=None, residual_out=None, q=None, scale=None, rstd=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last dimension F.

    x, residual (..., F) float32 or bfloat16 with evenly spaced rows; weight (F,) float32.
    Returns RMSNorm(y in x's type or None, residual = s in x's type (None without a
    residual), q (..., F) float8_e4m3fn and scale (ceil(F / 128), rows) float32 with fp8 (y in 8
    bits, as fp8_matmul reads it), rstd (rows,) float32 if wanted). residual_out may be
    residual (in place)."""
    dev = _device(x, "x")
    dt = _dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have a last dimension")
    F = x.shape[-1]
    rows = _rows(x.shape[:-1])
    sx = _row_stride(x, "x", x.dtype, x.shape, dev)
    sr = 0 if residual is None else _row_stride(residual, "residual", x.dtype, x.shape, dev)
    _check(weight, "weight", torch.float32, (F,), dev)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without a residual")
    y = _out(y, "y", x.dtype, x.shape, dev, want_y)
    residual_out = _out(residual_out, "residual_out", x.dtype, x.shape, dev, residual is not None)
    q = _out(q, "q", torch.float8_e4m3fn, x.shape, dev, fp8)
    scale = _out(scale, "scale", torch.float32, (-(-F // 128), rows), dev, q is not None)
    rstd = _out(rstd, "rstd", torch.float32, (rows,), dev, want_rstd)
    _call("ssd_rms_norm", dev, _ptr(x), sx, _ptr(residual), sr, _ptr(weight), dt, rows, F, float(eps),
          _ptr(y), _ptr(residual_out), _ptr(q), _ptr(scale), _ptr(rstd))
    return RMSNorm(y, residual_out, q, scale, rstd)


def rms_norm_backward(s, weight, rstd, grad_y, grad_residual=None, grad_x=None, grad_weight=None,
                      workspace=None):
    """Gradients of sum(grad_y * y) + sum(grad_residual * s) for rms_norm: s is its residual
    output (its x, where it had no residual), rstd (rows,) as it returned it. Returns
    (grad_x, grad_weight): grad_x (..., F) in s's type is the gradient of x and of residual,
    grad_weight (F,) float32."""
    dev = _device(s, "s")
    dt = _dtype(s, "s")
    if s.dim() < 1:
        raise ValueError("s must have a last dimension")
    F = s.shape[-1]
    rows = _rows(s.shape[:-1])
    ss = _row_stride(s, "s", s.dtype, s.shape, dev)
    sg = _row_stride(grad_y, "grad_y", s.dtype, s.shape, dev)
    sr = 0 if grad_residual is None else _row_stride(grad_residual, "grad_residual", s.dtype, s.shape, dev)
    _check(weight, "weight", torch.float32, (F,), dev)
    _check(rstd, "rstd", torch.float32, (rows,), dev)
    grad_x = _out(grad_x, "grad_x", s.dtype, s.shape, dev)
    grad_weight = _out(grad_weight, "grad_weight", torch.float32, (F,), dev)
    ws, size = _workspace(workspace, _entry("ssd_rms_norm_backward_workspace_bytes")(rows, F), dev)
    _call("ssd_rms_norm_backward", dev, _ptr(s), ss, _ptr(weight), _ptr(rstd), _ptr(grad_y), sg,
          _ptr(grad_residual), sr, dt, rows, F, _ptr(grad_x), _ptr(grad_weight), _ptr(ws), size)
    return grad_x, grad_weight


def _fp8_stride(t, name, shape, dev):
    return _row_stride(t, name, torch.float8_e4m3fn, shape, dev)


def fp8_quantise(x, block_rows: int = 1, transpose: bool = False, q=None, scale=None):
    """8-bit values (float8_e4m3fn) of x with a float32 scale per block of 128: scale = max |v| /
    448 over the block (at least 2^-126), q = v / scale. x (..., K) float32 or bfloat16 with
    evenly spaced rows, its leading dimensions taken as R rows.

    block_rows 1: 1 x 128 blocks, scale (ceil(K / 128), R); 128: 128 x 128 blocks, scale
    (ceil(R / 128), ceil(K / 128)). With transpose the same of x turned: q (K, R).
    Returns (q, scale). q's rows start on multiples of 16 bytes (K is padded in memory, not in
    shape), as fp8_matmul reads them fastest."""
    dev = _device(x, "x")
    dt = _dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have a last dimension")
    cols = x.shape[-1]
    rows = _rows(x.shape[:-1])
    sx = _row_stride(x, "x", x.dtype, x.shape, dev)
    R, K = (cols, rows) if transpose else (rows, cols)
    shape = (cols, rows) if transpose else tuple(x.shape)
    if q is None:
        wide = -(-K // 16) * 16
        q = torch.empty(shape[:-1] + (wide,), dtype=torch.float8_e4m3fn, device=dev)[..., :K]
    sq = _fp8_stride(q, "q", shape, dev)
    blocks = (-(-K // 128), R) if block_rows == 1 else (-(-R // 128), -(-K // 128))
    scale = _out(scale, "scale", torch.float32, blocks, dev)
    _call("ssd_fp8_quantise", dev, _ptr(x), sx, dt, rows, cols, int(block_rows), int(bool(transpose)),
          _ptr(q), sq, _ptr(scale))
    return q, scale


def fp8_matmul_workspace_bytes(M, N, K, block_rows=128, out_dtype=torch.bfloat16, rows_on_16=True) -> int:
    return int(_entry("ssd_fp8_matmul_workspace_bytes")(M, N, K, int(block_rows), _DTYPES[out_dtype], int(rows_on_16)))


def gated_scan_workspace_bytes(B, T, C, dtype, backward=False) -> int:
    name = "ssd_gated_scan_backward_workspace_bytes" if backward else "ssd_gated_scan_workspace_bytes"
    return int(_entry(name)(B, T, C, _DTYPES[dtype]))


def rms_norm_backward_workspace_bytes(rows, F) -> int:
    return int(_entry("ssd_rms_norm_backward_workspace_bytes")(rows, F))


def fp8_matmul(a, a_scale, b, b_scale, block_rows: int = 128, out_dtype=torch.bfloat16, out=None,
               workspace=None):
    """out[..., n] = sum over k of (a a_scale)[..., k] (b b_scale)[n, k], both operands 8-bit with a
    scale per block of 128 k. a (..., K) float8_e4m3fn with a_scale (ceil(K / 128), rows) (1 x 128
    blocks); b (N, K) with b_scale (ceil(N / 128), ceil(K / 128)) for block_rows 128, or
    (ceil(K / 128), N) for block_rows 1. Rows evenly spaced. Returns out (..., N) bfloat16 or
    float32; sums are float32."""
    dev = _device(a, "a")
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32 or bfloat16, got %s" % out_dtype)
    if a.dim() < 1 or not isinstance(b, torch.Tensor) or b.dim() != 2:
        raise ValueError("a must be (..., K) and b (N, K)")
    K = a.shape[-1]
    N = b.shape[0]
    M = _rows(a.shape[:-1])
    sa = _fp8_stride(a, "a", a.shape, dev)
    sb = _fp8_stride(b, "b", (N, K), dev)
    kb = -(-K // 128)
    _check(a_scale, "a_scale", torch.float32, (kb, M), dev)
    _check(b_scale, "b_scale", torch.float32, (kb, N) if block_rows == 1 else (-(-N // 128), kb), dev)
    shape = tuple(a.shape[:-1]) + (N,)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    so = _row_stride(out, "out", out_dtype, shape, dev)
    dt = _DTYPES[out_dtype]
    pa, pb = a.data_ptr(), b.data_ptr()
    on16 = int((pa | pb | sa | sb) % 16 == 0 and sa < 1 << 24 and sb < 1 << 24)
    ws, size = _workspace(workspace, fp8_matmul_workspace_bytes(M, N, K, block_rows, out_dtype, on16), dev)
    _call("ssd_fp8_matmul", dev, pa, sa, _ptr(a_scale), pb, sb, _ptr(b_scale), M, N, K,
          int(block_rows), dt, _ptr(out), so, _ptr(ws), size)
    return out
