"""The norms around a block: float64 definitions with bounds of what float32 arithmetic can make of them (U is
half a unit of float32, as in operators_ref), and the cases that the emulator and the GPU run alike (test-only).
Each case takes a `run` with the functions of block_norm_harness (numpy in, numpy out)."""

import numpy as np

import operators_ref as ref
from operators_ref import U

NAN = float("nan")


def _act(z):
    s = ref.sigmoid(z)
    return z * s, s, s * (1 + z * (1 - s))


# A sum of D (F) squares or products takes at most 32 additions in a lane and 16 across lanes and waves, or, through
# shared memory, 8 in a lane, 64 (F = 8192 values of one head in groups of eight by sixteen lanes) and 4: 80 U of the
# sum of magnitudes; half of it in rstd, with the division, eps and the root: 44 U. A sigmoid is good to 30 U
# for |z| <= 6 (operators_ref), 1 - sigmoid to 31 U of 1.
SUM, ROOT, GATE = 80 * U, 44 * U, 30 * U


def gated(x, z, w, D, eps):
    R, F = x.shape
    h = x.reshape(R, -1, D)
    rstd = 1 / np.sqrt((h * h).mean(2) + eps)
    y = (h * rstd[..., None] * w).reshape(R, F) * _act(z)[0]
    return (y, rstd), ((ROOT + GATE + 6 * U) * np.abs(y), ROOT * rstd)


def gated_backward(x, z, w, rstd, gy):
    """rstd as handed in."""
    R, F = x.shape
    D = F // rstd.shape[1]
    heads = lambda v: v.reshape(R, -1, D)  # noqa: E731
    r = rstd[..., None]
    n, zs, g = heads(x) * r, heads(z), heads(gy)
    act, sig, slope = _act(zs)
    gn = g * act
    b = gn * w
    mean, size = (b * n).mean(2, keepdims=True), np.abs(b * n).mean(2, keepdims=True)
    gx = r * (b - n * mean)
    gx_err = r * ((GATE + 8 * U) * np.abs(b) + np.abs(n) * (SUM + GATE + 10 * U) * size)
    gz = g * n * w * slope
    # sigmoid (1 + z (1 - sigmoid)): off by GATE of itself and sigmoid |z| 33 U
    gz_err = np.abs(g * n * w) * ((GATE + 8 * U) * np.abs(slope) + sig * (33 * U * np.abs(zs) + 4 * U))
    gw, gw_size = (gn * n).sum((0, 1)), np.abs(gn * n).sum((0, 1))
    flat = lambda v: v.reshape(R, F)  # noqa: E731
    # each product joins a chain of at most R rows, F / D heads and 80 more sums
    return (flat(gx), flat(gz), gw), (flat(gx_err), flat(gz_err), (GATE + U * (R + F // D + 90)) * gw_size)


def block(x, res, w1, w2, alpha, eps):
    r1 = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    add = alpha * w1 * x * r1
    s = res + add
    s_err = (ROOT + 4 * U) * np.abs(add) + U * np.abs(s)
    r2 = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    # the root's argument is off by the sum's own and by 2 |s| ds
    r2_err = r2 * (ROOT + (np.abs(s) * s_err).mean(1, keepdims=True) * r2 * r2)
    y = s * r2 * w2
    y_err = np.abs(w2) * (s_err * r2 + np.abs(s) * r2_err) + 4 * U * np.abs(y)
    return (y, s, r1[:, 0], r2[:, 0]), (y_err, s_err, ROOT * r1[:, 0], r2_err[:, 0])


def block_backward(x, s, w1, w2, r1, r2, alpha, gy, gs):
    R = len(x)
    r1, r2 = r1[:, None], r2[:, None]
    m, n, base = s * r2, x * r1, np.zeros_like(s) if gs is None else gs
    g = gy * w2
    mean, size = (g * m).mean(1, keepdims=True), np.abs(g * m).mean(1, keepdims=True)
    gres = base + r2 * (g - m * mean)
    err = U * 4 * np.abs(base) + r2 * (8 * U * np.abs(g) + np.abs(m) * (SUM + 10 * U) * size)
    a, a_err = alpha * gres, np.abs(alpha) * (err + 2 * U * np.abs(gres))
    b, b_err = a * w1, np.abs(w1) * a_err + 2 * U * np.abs(a * w1)
    mean, size = (b * n).mean(1, keepdims=True), np.abs(b * n).mean(1, keepdims=True)
    gx = r1 * (b - n * mean)
    gx_err = r1 * (b_err + 8 * U * np.abs(b) + np.abs(n) * ((SUM + 10 * U) * size + (b_err * np.abs(n)).mean(1, keepdims=True)))
    chain = U * (R + 90)
    return ((gx, gres, (a * n).sum(0), (gy * m).sum(0)),
            (gx_err, err, (a_err * np.abs(n)).sum(0) + chain * np.abs(a * n).sum(0), chain * np.abs(gy * m).sum(0)))


# rows, heads, D, kind, padding between rows: whole lanes and not, one value past a lane, every width of row
GATED = [
    (1, 1, 8, "f32", 0),
    (3, 5, 9, "bf16", 1),
    (5, 16, 64, "bf16", 0),
    (2, 3, 43, "f32", 3),
    (9, 4, 128, "bf16", 0),
    (18, 2, 16, "f32", 0),
    (4, 10, 100, "bf16", 8),
    (3, 32, 32, "f32", 0),
    (2, 1, 1000, "bf16", 2),
    (3, 17, 120, "f32", 0),
    (2, 37, 77, "bf16", 1),
    (2, 8, 512, "bf16", 0),
    (2, 32, 256, "f32", 0),
    (2, 63, 130, "bf16", 0),
    (2, 128, 128, "bf16", 0),
    (2, 2, 8192, "f32", 0),
    (2, 1024, 9, "bf16", 0),
    (33, 8, 8, "bf16", 0),
]


def _rows(g, rows, F, kind, scale=1.0):
    return ref.rounded(np.clip(scale * g.standard_normal((rows, F)), -6, 6), kind)


def _weight(g, n):
    return np.float32(1 + 0.3 * g.standard_normal(n)).astype(np.float64)


def run_gated(run, rows, H, D, kind, pad):
    g = np.random.default_rng(rows * H + D)
    x, z, w = _rows(g, rows, H * D, kind), _rows(g, rows, H * D, kind, 1.5), _weight(g, D)
    (y, rstd), (ey, er) = gated(x, z, w, D, 1e-6)
    got = run.gated_norm(x, z, w, 1e-6, kind, pad=pad)
    ref.close(got["y"], y, ey, kind, "y")
    ref.close(got["rstd"], rstd, er, "f32", "rstd")
    ref.check_quantised(y, ey, got["q"], got["scale"].astype(np.float64), 1)
    only = run.gated_norm(x, z, w, 1e-6, kind, y=False, pad=pad)
    assert np.array_equal(only["q"], got["q"]) and np.array_equal(only["scale"], got["scale"])
    assert np.array_equal(run.gated_norm(x, z, w, 1e-6, kind, fp8=False, pad=pad)["y"], got["y"])


def run_gated_backward(run, rows, H, D, kind, pad):
    g = np.random.default_rng(rows * H + D + 1)
    x, z, w = _rows(g, rows, H * D, kind), _rows(g, rows, H * D, kind, 1.5), _weight(g, D)
    gy = _rows(g, rows, H * D, kind)
    rstd = np.float32(1 / np.sqrt((x.reshape(rows, H, D) ** 2).mean(2) + 1e-6)).astype(np.float64)
    want, err = gated_backward(x, z, w, rstd, gy)
    got = run.gated_norm_backward(x, z, w, rstd, gy, kind, pad=pad)
    for name, a, b, e, k in zip(("x", "gate", "weight"), got, want, err, (kind, kind, "f32")):
        ref.close(a, b, e, k, name)


# rows, F, kind, gradient of the residual stream, padding between rows
BLOCK = [
    (1, 1, "f32", True, 0),
    (3, 7, "bf16", True, 1),
    (5, 128, "bf16", False, 0),
    (2, 129, "f32", True, 3),
    (9, 513, "bf16", True, 0),
    (6, 1024, "bf16", True, 8),
    (3, 2047, "bf16", True, 0),
    (2, 4096, "f32", False, 0),
    (3, 5000, "bf16", True, 0),
    (2, 8193, "f32", True, 0),
    (2, 16384, "bf16", True, 0),
    (18, 65, "bf16", True, 0),
]


def run_block(run, rows, F, kind, stream, pad):
    g = np.random.default_rng(rows * F)
    x, res = _rows(g, rows, F, kind), _rows(g, rows, F, kind, 2.0)
    w1, w2, alpha = _weight(g, F), _weight(g, F), float(np.float32(0.3))
    (y, s, r1, r2), (ey, es, e1, e2) = block(x, res, w1, w2, alpha, 1e-6)
    got = run.block_norm(x, res, w1, w2, alpha, 1e-6, kind, pad=pad)
    for name, a, b, e, k in (("y", got["y"], y, ey, kind), ("s", got["s"], s, es, kind), ("post", got["post"], r1, e1, "f32"),
                             ("pre", got["pre"], r2, e2, "f32")):
        ref.close(a, b, e, k, name)
    ref.check_quantised(y, ey, got["q"], got["scale"].astype(np.float64), 1)
    only = run.block_norm(x, res, w1, w2, alpha, 1e-6, kind, y=False, pad=pad, in_place=True)
    assert all(np.array_equal(only[k], got[k]) for k in ("q", "scale", "s", "post", "pre"))
    assert np.array_equal(run.block_norm(x, res, w1, w2, alpha, 1e-6, kind, fp8=False, pad=pad)["y"], got["y"])


def run_block_backward(run, rows, F, kind, stream, pad):
    g = np.random.default_rng(rows * F + 1)
    x, s, gy = _rows(g, rows, F, kind), _rows(g, rows, F, kind, 2.0), _rows(g, rows, F, kind)
    gs = _rows(g, rows, F, kind) if stream else None
    w1, w2, alpha = _weight(g, F), _weight(g, F), float(np.float32(-0.7))
    r1, r2 = (np.float32(1 / np.sqrt((v * v).mean(1) + 1e-6)).astype(np.float64) for v in (x, s))
    want, err = block_backward(x, s, w1, w2, r1, r2, alpha, gy, gs)
    got = run.block_norm_backward(x, s, w1, w2, r1, r2, alpha, gy, gs, kind, pad=pad)
    for name, a, b, e, k in zip(("x", "residual", "post_weight", "pre_weight"), got, want, err, (kind, kind, "f32", "f32")):
        ref.close(a, b, e, k, name)


def rows_apart(run):
    """A row of zeros, one with a NaN, one with gates far from 0: what each makes of itself, and the others' bits."""
    g = np.random.default_rng(5)
    x, z, w = _rows(g, 6, 96, "f32"), _rows(g, 6, 96, "f32"), _weight(g, 24)
    clean = run.gated_norm(x, z, w, 1e-6, "f32")
    x[1] = 0
    x[2, 30] = NAN
    z[3, :8], z[3, 8:16] = -200, 200
    got = run.gated_norm(x, z, w, 1e-6, "f32")
    assert (got["y"][1] == 0).all() and (got["q"][1] & 0x7f == 0).all()
    assert np.isnan(got["y"][2, 24:48]).all() and np.isfinite(got["y"][2, :24]).all() and np.isfinite(got["y"][2, 48:]).all()
    assert (got["y"][3, :8] == 0).all()
    n = x[3, 8:16] * clean["rstd"][3, 0] * w[8:16]
    assert np.abs(got["y"][3, 8:16] - 200 * n).max() <= 200 * 50 * U * np.abs(n).max()
    for r in (0, 4, 5):
        assert np.array_equal(got["y"][r], clean["y"][r]) and np.array_equal(got["q"][r], clean["q"][r])
    b = run.block_norm(x, z * 0 + 1, np.ones(96), np.ones(96), 0.5, 1e-6, "f32")
    assert np.isnan(b["y"][2]).all() and (b["s"][1] == 1).all() and np.isfinite(b["y"][[0, 1, 3, 4, 5]]).all()
