"""Calls at the edges of what the operators around the scan allow, which the emulator and the GPU
run alike (test-only). Each takes a `run` with the functions of ops_emu_harness (numpy in, numpy
out)."""

import numpy as np

import operators_ref as ref


def _same(a, b):
    assert all(np.array_equal(p, q) for p, q in zip(a, b) if p is not None)


def gated_lengths_lowest(run):
    """The lowest length that there is counts as 0, in the walk, in one tile and over segments."""
    low = -2 ** 31
    for B, T, C in ((3, 5, 6), (3, 70, 6), (3, 700, 6)):
        x, gi, gr, lam, init, _ = ref.gated_case(B, T, C, "f32", T, state=True)
        gh, gf = np.random.default_rng(T).standard_normal((B, T, C)), np.ones((B, C))
        got, want = [], []
        for lengths, out in (([low, T, low + 1], got), ([0, T, 0], want)):
            n = np.array(lengths, np.int32)
            out += run.gated(x, gi, gr, lam, 8.0, "f32", init=init, lengths=n, states=True)
            out += run.gated_backward(x, gi, gr, lam, 8.0, "f32", out[2], gh, gfinal=gf, lengths=n)
        _same(got, want)
        assert np.array_equal(got[1][0], init[0]) and not got[0][0].any()


def gated_adjoint_takes_the_decays_of_the_forward(run):
    """One state that only decays, and one gradient that comes back to it over several segments:
    with a = 1 (a closed decay gate) at every token but one or two, their product is rounded once at most
    and both directions give the same bits."""
    for kind, T, C, tokens in (("f32", 1000, 130, (600,)), ("f32", 1000, 130, (450, 900)), ("bf16", 1500, 256, (700, 1400)),
                               ("bf16", 1500, 255, (5, 1499))):
        g = np.random.default_rng(T)
        zero, one = np.zeros((1, T, C)), np.ones((1, C))
        gr = np.full((1, T, C), -200.0)
        gr[:, tokens] = ref.rounded(g.standard_normal((1, len(tokens), C)), kind)
        full = 1 - np.exp(g.uniform(np.log(1e-6), np.log(0.7), C))
        lam = np.float32(np.log(np.expm1(-np.log(full) / 8))).astype(np.float64)
        _, final, states = run.gated(zero, zero, gr, lam, 8.0, kind, init=one, states=True)
        got = run.gated_backward(zero, zero, gr, lam, 8.0, kind, states, zero, gfinal=one)
        assert (final < 1).any()
        assert np.array_equal(got[4], final), (kind, tokens, np.abs(got[4] - final).max())


def gated_decays_beyond_float32(run):
    """decay_scale * softplus(lam) past the largest float, large states and gradients: a = 0 and the gradients
    by the decay are 0, not infinity times zero; a closed gate (r = 0) still keeps the state."""
    B, T, C = 2, 6, 8
    for kind in ("f32", "bf16"):
        for k, lam_at in ((1e30, 1e9), (1e30, 10.0), (8.0, 3e38), (8.0, np.inf)):
            g = np.random.default_rng(3)
            x, gi, gr, gh = (ref.rounded(g.standard_normal((B, T, C)), kind) for _ in range(4))
            lam, init = np.full(C, lam_at), np.full((B, C), 1e10)
            i = ref.sigmoid(gi)
            h, final, states = run.gated(x, gi, gr, lam, k, kind, init=init, states=True)
            bar = 30 * ref.U * np.abs(x) + ref.HALF[kind] * np.abs(i * x)
            assert (np.abs(h - i * x) <= bar).all()     # a = 0, m = 1
            gx, ggi, ggr, glam, ginit = run.gated_backward(x, gi, gr, lam, k, kind, states, gh, gfinal=np.ones((B, C)))
            assert not ggr.any() and not glam.any() and not ginit.any(), (kind, k, lam_at)
            last = gh + np.concatenate([np.zeros((B, T - 1, C)), np.ones((B, 1, C))], 1)
            assert (np.abs(gx - i * last) <= 40 * ref.U * np.abs(last) + ref.HALF[kind] * np.abs(i * last)).all()
            closed = np.full((B, T, C), -np.inf)
            assert np.array_equal(run.gated(x, gi, closed, lam, k, kind, init=init)[1], np.float32(init))


def gated_lowest_lam(run):
    """grad_lam where exp(-lam) passes the largest float and softplus(lam) = exp(lam) is denormal: sigmoid /
    softplus is 1, down to where both are 0. A large state makes the sum a number: -k sigmoid(lam) sum r g h.
    softplus and l are off by 4 units of the denormals, 2^-149, at most; the rest as elsewhere (below 100 U)."""
    T, k = 70, 8.0
    lam = np.array([-60.0, -85, -88, -89, -90, -93, -95, -200])
    C = len(lam)
    gr = ref.rounded(np.random.default_rng(4).standard_normal((1, T, C)), "f32")
    zero, init = np.zeros((1, T, C)), np.float32(np.full((1, C), 1e30)).astype(np.float64)
    states = run.gated(zero, zero, gr, lam, k, "f32", init=init, states=True)[2]
    got = run.gated_backward(zero, zero, gr, lam, k, "f32", states, zero, gfinal=np.ones((1, C)))[3]
    want = -k * np.exp(lam) * ref.sigmoid(gr).sum((0, 1)) * init[0]     # a is 1, g is 1, sigmoid(lam) exp(lam)
    rel = 100 * ref.U + 4 * 2.0 ** -149 / np.exp(lam)
    ok = np.abs(got - want) <= rel * np.abs(want)
    assert ok[:-1].all() and abs(got[-1]) <= 1e-12, got / want


def norm_of_small_rows(run):
    """Rows whose mean square is denormal, without an epsilon: still normed. Each square and the mean
    are off by half a unit of the denormals, 2^-150, so v by 2^-149 and rstd by 2^-150 / v. A row of zeros has
    no norm; rows next to it do not see it."""
    F = 200
    g = np.random.default_rng(5)
    x = g.standard_normal((7, F)) * np.array([1e-15, 1e-18, 2e-19, 3e-20, 1e-20, 3e-21, 0.0])[:, None]
    w = np.float32(1 + 0.3 * g.standard_normal(F)).astype(np.float64)
    for kind in ("f32", "bf16"):
        v = ref.rounded(x, kind)
        got = run.norm(v, None, w, 0.0, kind, fp8=False)
        mean = (v[:6] ** 2).mean(1)
        rel = 40 * ref.U + 2.0 ** -150 / mean
        want = 1 / np.sqrt(mean)
        assert (np.abs(got["rstd"][:6] - want) <= rel * want).all(), got["rstd"][:6] / want
        y = v[:6] * want[:, None] * w
        assert (np.abs(got["y"][:6] - y) <= (rel[:, None] + 4 * ref.U + ref.HALF[kind]) * np.abs(y)).all()
        assert np.isnan(got["y"][6]).all() and np.isposinf(got["rstd"][6])


def _over(v, scale):
    """v / scale in float32, rounded once more to the nearest e4m3 value (ties to even), as values."""
    t = (np.float32(v) / np.float32(scale)).astype(np.float64)
    _, e = np.frexp(t)
    step = 2.0 ** (np.maximum(e - 1, -6) - 3)
    return np.rint(t / step) * step


def quantise_is_a_division(run):
    """Scales and values bit for bit those of float32 divisions: bfloat16 values often lie on a border of
    two e4m3 values, where half a unit decides."""
    for kind in ("bf16", "f32"):
        for block_rows, turn in ((1, False), (1, True), (128, False), (128, True)):
            x = ref.rounded(np.random.default_rng(7).standard_normal((256, 384)), kind)
            q, scale = run.quantise(x, kind, block_rows, turn)
            v = x.T if turn else x
            R, K = v.shape
            top = np.abs(v).reshape(R // block_rows, block_rows, K // 128, 128).max((1, 3))
            want = np.float32(top) / np.float32(448)
            assert np.array_equal(scale, want.T if block_rows == 1 else want)
            full = np.repeat(np.repeat(want, block_rows, 0), 128, 1)
            assert np.array_equal(ref.E4M3[q], _over(v, full)), (kind, block_rows, turn)


# One value's largest relative errors in U for gates of any size, as operators_ref derives them for gates
# within 6: sigmoid(v) is off by 3 |v| + 5, l by 8 more; a by |l| (that + 3) + 2; 1 - a from the series (l below
# 1/16) by 8 and l's error, else by a's times a / (1 - a); its root by half of that and 4.
def _gate_errors(gi, gr, l, a):
    e_i, e_r = 3 * np.abs(gi) + 5, 3 * np.abs(gr) + 5
    e_l = e_r + 8
    e_a = np.abs(l) * (e_l + 3) + 2
    near, far = (8 + e_l) / 2, e_a * a / np.maximum(1 - a, 1e-3) / 2
    border = np.abs(-l - 0.0625) < 1e-3
    e_m = 4 + np.where(border, np.maximum(near, far), np.where(-l < 0.0625, near, far))
    return e_i, e_r, e_l, e_a, e_m


def gated_extreme_gates(run):
    """Gates saturated at both ends, lam from where a = 1 to where it is 0, no decay at all: one token from a
    given state, and its gradients, against float64."""
    for kind in ("f32", "bf16"):
        g = np.random.default_rng(8)
        at = np.array([-80.0, -30, -12, -3, 0, 3, 12, 30, 80])
        gi, gr = (ref.rounded(v.reshape(1, 1, -1), kind) for v in np.meshgrid(at, at))
        for k in (0.0, 1e-3, 8.0):
            for lam_at in (-20.0, -5, 0, 5, 50):
                C = gi.shape[2]
                x, gh = (ref.rounded(g.standard_normal((1, 1, C)), kind) for _ in range(2))
                init, gf = (np.float32(g.standard_normal((1, C))).astype(np.float64) for _ in range(2))
                lam = np.full(C, lam_at)
                k = float(np.float32(k))
                i, r, l, a, m = ref.gates(gi, gr, lam, k)
                e_i, e_r, e_l, e_a, e_m = _gate_errors(gi, gr, l, a)
                u = m * i * x
                want = a * init[:, None] + u
                err = ref.U * ((e_a + 3) * a * np.abs(init[:, None]) + (e_m + e_i + 4) * np.abs(u) + 2 * np.abs(want))
                # below 2^-126 the hardware's results and roots' arguments may be flushed to zero
                flush = 2.0 ** -63 * np.abs(x) * (1 - a * a < 2.0 ** -125) + 2.0 ** -120
                h, final, states = run.gated(x, gi, gr, lam, k, kind, init=init, states=True)
                ref.close(h, want, err + flush, kind, "h")
                ref.close(final, want[:, 0], (err + flush)[:, 0], "f32", "final")
                gx, ggi, ggr, glam, ginit = run.gated_backward(x, gi, gr, lam, k, kind, states, gh, gfinal=gf)
                adj = gh + gf[:, None]
                ratio = np.where(m > 0, l / np.where(m > 0, m, 1), 0)
                w_gx = adj * m * i
                rel = (e_m + e_i + 6) * ref.U
                ref.close(gx, w_gx, rel * np.abs(w_gx) + np.abs(adj) * flush, kind, "grad x")
                w_ggi = w_gx * x * (1 - i)      # 1 - i is off by i's error and half a unit of 1
                one_i = (e_i * i + 1) * ref.U
                ref.close(ggi, w_ggi, np.abs(w_gx * x) * (rel * (1 - i) + 2 * one_i + 4 * ref.U) + np.abs(adj * x) * flush, kind,
                          "grad input_gate")
                one, two = adj * a * init[:, None] * l, adj * i * x * a * a * ratio
                e_err = ref.U * ((e_a + e_l + 8) * np.abs(one) + (e_i + 2 * e_a + e_l + e_m + 12) * np.abs(two)) + \
                    np.abs(adj * x) * flush
                e = one - two
                one_r = (e_r * r + 1) * ref.U
                ref.close(ggr, e * (1 - r), e_err * (1 - r) + (np.abs(one) + np.abs(two)) * (2 * one_r + 4 * ref.U), kind,
                          "grad decay_gate")
                factor = ref.sigmoid(lam) / ref.softplus(lam)
                ref.close(glam, factor * e[0, 0], factor * (e_err + 20 * ref.U * (np.abs(one) + np.abs(two)))[0, 0], "f32", "grad lam")
                # a gf + (a gh): each product is rounded for itself, before the sum, which may cancel
                parts = np.abs(gh) + np.abs(gf[:, None])
                ref.close(ginit, (a * adj)[:, 0], (ref.U * (e_a + 4) * a * parts + 2.0 ** -120)[:, 0], "f32", "grad init")


ALL = {f.__name__: f for f in (gated_lengths_lowest, gated_adjoint_takes_the_decays_of_the_forward,
                               gated_decays_beyond_float32, gated_lowest_lam, norm_of_small_rows,
                               quantise_is_a_division, gated_extreme_gates)}
