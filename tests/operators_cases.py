"""Cases of the operators around the scan that the emulator and the GPU run alike (test-only).
Each takes a `run` with the functions of ops_emu_harness (numpy in, numpy out)."""

import numpy as np

import operators_ref as ref

NAN = float("nan")

# B, T, C, kind, state, lengths, padding between rows
GATED = [
    (1, 1, 1, "f32", True, None, 0),
    (3, 1, 70, "bf16", True, [1, 0, 1], 2),
    (2, 2, 3, "bf16", False, None, 1),
    (2, 63, 5, "f32", True, [63, 0], 0),
    (1, 64, 64, "bf16", False, None, 0),
    (2, 65, 129, "bf16", True, [65, 64], 3),
    (1, 200, 66, "f32", True, None, 0),
    (2, 333, 7, "bf16", True, [1, 333], 0),
    (1, 700, 65, "f32", True, [650], 1),     # several segments, the end inside the last
    (1, 1025, 131, "bf16", False, None, 0),
    (3, 600, 2, "bf16", True, [0, 300, 600], 0),
    (2, 8, 65, "bf16", True, [8, 3], 0),     # the longest that is walked by lanes, and one more
    (2, 9, 65, "bf16", True, [9, 3], 0),
    (1, 4700, 3, "f32", True, [4650], 0),    # more segments than waves that fold them
]


def gated(run, B, T, C, kind, state, lengths, pad):
    x, gi, gr, lam, init, n = ref.gated_case(B, T, C, kind, seed=B * 1000 + T, state=state, lengths=lengths)
    want, err = ref.gated(x, gi, gr, lam, 8.0, init, n)
    if n is not None:  # what lies in the padding is not read
        dead = np.arange(T)[None, :] >= n[:, None]
        x, gi, gr = (np.where(dead[..., None], v, w) for v, w in ((NAN, x), (np.inf, gi), (-np.inf, gr)))
    h, final, states = run.gated(x, gi, gr, lam, 8.0, kind, init=init, lengths=n, states=True, pad=pad)
    ref.close(h, want[0], err[0], kind, "h")
    ref.close(final, want[1], err[1], "f32", "final")
    ref.close(states, want[2], err[2], "f32", "states")
    if init is not None:
        again = run.gated(x, gi, gr, lam, 8.0, kind, init=init, lengths=n, pad=pad, in_place=True)
        assert np.array_equal(again[0], h) and np.array_equal(again[1], final)


def gated_backward(run, B, T, C, kind, state, lengths, pad):
    x, gi, gr, lam, init, n = ref.gated_case(B, T, C, kind, seed=B * 1000 + T + 1, state=True, lengths=lengths)
    g = np.random.default_rng(T)
    gh = ref.rounded(g.standard_normal((B, T, C)), kind)
    gf = np.float32(g.standard_normal((B, C))).astype(np.float64) if state else None
    (_, _, states), (_, _, states_err) = ref.gated(x, gi, gr, lam, 8.0, init, n)
    want, err = ref.gated_backward(x, gi, gr, lam, 8.0, init, gh, gf, n)
    if n is not None:
        dead = (np.arange(T)[None, :] >= n[:, None])[..., None]
        x, gi, gr, gh = (np.where(dead, NAN, v) for v in (x, gi, gr, gh))
    got = run.gated_backward(x, gi, gr, lam, 8.0, kind, states, gh, gfinal=gf, lengths=n, pad=pad)
    for name, v, w, e, k in zip(("x", "input_gate", "decay_gate", "lam", "init"), got, want, err,
                                (kind, kind, kind, "f32", "f32")):
        ref.close(v, w, e, k, name)


def gated_lengths_clamped(run):
    """Lengths below 0 and past T are taken as 0 and as T."""
    x, gi, gr, lam, init, _ = ref.gated_case(3, 70, 6, "f32", 5, state=True)
    a = run.gated(x, gi, gr, lam, 8.0, "f32", init=init, lengths=np.array([-3, 75, 2 ** 31 - 1], np.int32))
    b = run.gated(x, gi, gr, lam, 8.0, "f32", init=init, lengths=np.array([0, 70, 70], np.int32))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def gated_empty_row_infinite(run):
    """A row without tokens hands its final state's gradient to the initial state and leaves the
    others' gradients alone, be it infinite."""
    x, gi, gr, lam, init, _ = ref.gated_case(2, 70, 6, "f32", 6, state=True)
    n = np.array([70, 0], np.int32)
    states = ref.gated(x, gi, gr, lam, 8.0, init, n)[0][2]
    gf = np.ones((2, 6))
    want = run.gated_backward(x, gi, gr, lam, 8.0, "f32", states, x, gfinal=gf, lengths=n)
    gf[1] = np.inf
    got = run.gated_backward(x, gi, gr, lam, 8.0, "f32", states, x, gfinal=gf, lengths=n)
    assert all(np.array_equal(a, b) for a, b in zip(got[:4], want[:4]))
    assert np.array_equal(got[4][0], want[4][0]) and np.isposinf(got[4][1]).all()


# rows, F, kind, residual, padding between rows
NORM = [
    (1, 1, "f32", False, 0),
    (3, 7, "bf16", True, 1),
    (5, 128, "bf16", True, 0),
    (2, 129, "f32", True, 3),
    (9, 513, "bf16", True, 0),
    (4, 1000, "f32", False, 0),
    (6, 1024, "bf16", True, 8),
    (3, 2047, "bf16", True, 0),
    (2, 4096, "f32", True, 0),
    (3, 5000, "bf16", False, 0),
    (2, 16384, "bf16", True, 0),
    (2, 8193, "f32", True, 0),
    (18, 65, "bf16", True, 0),
]


def norm_inputs(rows, F, kind, residual, seed):
    g = np.random.default_rng(seed)
    x = ref.rounded(g.standard_normal((rows, F)), kind)
    res = ref.rounded(2 * g.standard_normal((rows, F)), kind) if residual else None
    w = np.float32(1 + 0.3 * g.standard_normal(F)).astype(np.float64)
    return g, x, res, w


def norm(run, rows, F, kind, residual, pad):
    _, x, res, w = norm_inputs(rows, F, kind, residual, rows * F)
    (y, s, rstd), (ey, es, er) = ref.norm(x, res, w, 1e-6)
    got = run.norm(x, res, w, 1e-6, kind, pad=pad)
    ref.close(got["y"], y, ey, kind, "y")
    ref.close(got["rstd"], rstd, er, "f32", "rstd")
    if residual:
        ref.close(got["s"], s, es, kind, "s")
    ref.check_quantised(y, ey, got["q"], got["scale"].astype(np.float64), 1)
    only = run.norm(x, res, w, 1e-6, kind, y=False, pad=pad, in_place=residual)
    assert np.array_equal(only["q"], got["q"]) and np.array_equal(only["scale"], got["scale"])
    if residual:
        assert np.array_equal(only["s"], got["s"])
    assert np.array_equal(run.norm(x, res, w, 1e-6, kind, fp8=False, pad=pad)["y"], got["y"])


def norm_backward(run, rows, F, kind, residual, pad):
    g, s, _, w = norm_inputs(rows, F, kind, residual, rows * F + 1)
    gy = ref.rounded(g.standard_normal((rows, F)), kind)
    gs = ref.rounded(g.standard_normal((rows, F)), kind) if residual else None
    rstd = np.float32(1 / np.sqrt((s * s).mean(1) + 1e-6)).astype(np.float64)
    (gx, gw), (ex, ew) = ref.norm_backward(s, w, rstd, gy, gs)
    got = run.norm_backward(s, w, rstd, gy, gs, kind, pad=pad)
    ref.close(got[0], gx, ex, kind, "grad_x")
    ref.close(got[1], gw, ew, "f32", "grad_weight")


# rows, cols, kind, padding of x's rows and of q's
QUANTISE = [
    (1, 1, "f32", 0, 0),
    (3, 5, "bf16", 1, 2),
    (7, 128, "bf16", 0, 0),
    (130, 130, "f32", 0, 6),
    (129, 300, "bf16", 4, 0),
    (256, 127, "bf16", 1, 1),
    (64, 1000, "f32", 0, 0),
    (300, 17, "bf16", 0, 15),
]


def quantise(run, rows, cols, kind, pad, q_pad, block_rows, turn):
    g = np.random.default_rng(rows * 1000 + cols)
    x = g.standard_normal((rows, cols)) * np.exp(3 * g.standard_normal((rows, 1)))
    x[:, cols // 2] = 0
    if rows > 4:
        x[3] = 0                        # whole blocks of zeros
        x[4] = np.float32(1e-39)        # and of values whose scale meets its floor
    x = ref.rounded(x, kind)
    q, scale = run.quantise(x, kind, block_rows, turn, pad=pad, q_pad=q_pad)
    v = x.T if turn else x
    # the floor of the scale: below 448 * 2^-126 a quotient of the smallest floats may be flushed
    ref.check_quantised(np.where(np.abs(v) < 2.0 ** -126, 0, v), np.where(np.abs(v) < 2.0 ** -126, np.abs(v), 0),
                        q, scale.astype(np.float64), block_rows)


def quantise_special(run, block_rows, turn):
    """An infinity or a NaN turns its own block into NaN and no other."""
    x = ref.rounded(np.random.default_rng(0).standard_normal((260, 260)), "bf16")
    clean = run.quantise(x, "bf16", block_rows, turn)
    x[5, 7], x[140, 250] = np.inf, np.nan
    q, scale = run.quantise(x, "bf16", block_rows, turn)
    v = x.T if turn else x
    with np.errstate(invalid="ignore"):
        got = scale.T if block_rows == 1 else scale
        got = np.repeat(np.repeat(got, block_rows, 0), 128, 1)[:260, :260] * ref.E4M3[q]
    bad = np.zeros_like(v, bool)
    for r, c in np.argwhere(~np.isfinite(v)):
        r0, c0 = r // block_rows * block_rows, c // 128 * 128
        bad[r0:r0 + block_rows, c0:c0 + 128] = True
    # with an infinity the scale is infinite: zero times it is NaN as well
    assert np.isnan(got[bad]).all()
    assert np.array_equal(q[~bad], clean[0][~bad]) and np.isfinite(got[~bad]).all()


# M, N, K, block_rows, out, paddings of a, b and out
MATMUL = [
    (1, 1, 1, 128, "f32", 0, 0, 0),
    (1, 5, 16, 1, "f32", 0, 0, 0),
    (3, 130, 129, 128, "bf16", 0, 0, 1),
    (1, 300, 256, 128, "bf16", 0, 0, 0),
    (7, 96, 640, 1, "f32", 16, 0, 0),
    (16, 64, 100, 1, "bf16", 12, 28, 0),
    (17, 257, 384, 128, "bf16", 0, 0, 0),
    (40, 33, 1000, 128, "f32", 0, 8, 3),
    (129, 140, 260, 1, "f32", 12, 12, 0),
    (130, 70, 2048, 128, "f32", 0, 0, 0),
    (260, 260, 200, 128, "bf16", 8, 8, 0),
    (70, 12, 2176, 1, "bf16", 0, 0, 0),
    (64, 48, 131, 1, "f32", 0, 0, 0),
    (65, 48, 131, 128, "bf16", 0, 0, 0),
]


def matmul_special(run, M, out):
    """A NaN in a row of a and one in a row of b come out in that row and that column only."""
    N, K = 40, 400
    a, sa, b, sb = matmul_inputs(M, N, K, 1, M)
    clean = run.matmul(a, sa, b, sb, 1, out)
    a[M // 2, 200], b[33, 399] = 0x7f, 0xff
    got = run.matmul(a, sa, b, sb, 1, out)
    bad = np.zeros((M, N), bool)
    bad[M // 2], bad[:, 33] = True, True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def matmul_inputs(M, N, K, block_rows, seed):
    g = np.random.default_rng(seed)
    a, b = (g.integers(0, 256, s, dtype=np.uint8) for s in ((M, K), (N, K)))
    a[(a & 127) == 127] ^= 1            # no NaN
    b[(b & 127) == 127] ^= 1
    kb = -(-K // 128)
    sa = np.float32(np.exp(g.standard_normal((kb, M))))
    sb = np.float32(np.exp(g.standard_normal((kb, N) if block_rows == 1 else (-(-N // 128), kb))))
    return a, sa, b, sb


def matmul(run, M, N, K, block_rows, out, a_pad, b_pad, out_pad, align=16):
    a, sa, b, sb = matmul_inputs(M, N, K, block_rows, M * N + K)
    want, err = ref.matmul(ref.E4M3[a], sa, ref.E4M3[b], sb, block_rows, out)
    got = run.matmul(a, sa, b, sb, block_rows, out, a_pad=a_pad, b_pad=b_pad, out_pad=out_pad, align=align)
    ref.close(got, want, err, out, "out")
