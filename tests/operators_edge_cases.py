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


ALL = {f.__name__: f for f in (gated_lengths_lowest, gated_adjoint_takes_the_decays_of_the_forward,
                               gated_decays_beyond_float32, gated_lowest_lam, norm_of_small_rows)}
