"""Further cases of the gated delta rule that the emulator and the GPU run alike (test-only), as delta_cases: each takes a
`run` with the functions of delta_emu_harness."""

import numpy as np

# B, Hv, Dk, Dv of every form of the walk: token by token (fewer than 9 tokens), few heads with 64 and with 128 features, and
# many heads by 64 and by 128 columns to a workgroup, most of whose rows are empty and cost nothing
HALFWAY = [(1, 2, 20, 18, 6), (1, 1, 64, 20, 64), (2, 1, 128, 17, 100), (97, 2, 64, 20, 64), (97, 2, 128, 33, 100),
           (97, 1, 128, 130, 100)]


def _rows(B, n):
    """Lengths: the first row's alone, or, with many rows, two of them."""
    lengths = np.zeros(B, np.int32)
    lengths[0], lengths[-1] = n, n
    return lengths


def halfway(run, B, Hv, Dk, Dv, T):
    """Outputs that lie 2^-20 above the middle of two bfloat16 numbers have to be the upper one: what makes them has 24 bits,
    whichever factor holds the last one. Everything is exact up to the rounding of o: keys are
    different unit vectors, so that a token's u is beta v."""
    x, up = 1 + 2.0 ** -8 + 2.0 ** -20, 1 + 2.0 ** -7
    n = _rows(B, T)
    live = n > 0
    k = np.zeros((B, T, 1, Dk))
    k[:, np.arange(T), 0, np.arange(T)] = 1.0
    last = np.zeros_like(k)     # the token before, at odd places
    at = np.arange(T) - np.arange(T) % 2
    last[:, np.arange(T), 0, at] = 1.0
    ones, none = np.ones((B, T, Hv)), np.zeros((B, T, Hv))
    v = np.ones((B, T, Hv, Dv))
    state = np.full((B, Hv, Dk, Dv), x)
    for what, q, beta, scale, init in (("state", k, none, 1.0, state), ("u", k, ones * x, 1.0, None), ("u", last, ones * x, 1.0, None),
                                       ("scale", last, ones, x, None), ("scale and state", k, none, x, state * 0 + 1)):
        o, final, _ = run.delta(q, k, v, none, beta, scale, "bf16", init=init, lengths=n)
        assert (o[live] == up).all(), (what, np.unique(o[live]))
        assert (o[~live] == 0).all(), what


# kind, B, Hv, Dv: few heads, many by 64 and by 128 columns to a workgroup
DECAYS = [("f32", 1, 1, 20), ("bf16", 1, 2, 16), ("f32", 97, 2, 20), ("bf16", 97, 2, 16), ("f32", 97, 1, 72), ("bf16", 97, 1, 72)]


def decays(run, kind, B, Hv, Dv):
    """A decay of many powers of two is right to a few units, not to a few units of its exponent. Token t writes a one into row
    t of the state, and what is left of it in the end, and of rows that held ones before, are single exponentials: off by 1
    unit (2^-23) in the hardware's, half a unit each in its correction and in two products."""
    T, Dk = 60, 64 if Dv <= 64 else 72
    r = np.random.default_rng(Dv + B)
    g = np.float32(-r.uniform(0.0, 2.6, (B, T, Hv))).astype(np.float64)   # down to e^-78 or so
    k = np.zeros((B, T, 1, Dk))
    q = np.zeros((B, T, 1, Dk))
    t = np.arange(T)
    k[:, t, 0, t] = 1.0
    q[:, t, 0, np.where(t % 2 == 0, t // 2, T)] = 1.0
    init = np.zeros((B, Hv, Dk, Dv))
    init[:, :, T:] = 1.0
    n = _rows(B, T)
    o, final, _ = run.delta(q, k, np.ones((B, T, Hv, Dv)), g, np.ones((B, T, Hv)), 1.0, kind, init=init, lengths=n)
    G = g.cumsum(1)
    want = np.exp(np.concatenate([G[:, -1:] - G, np.repeat(G[:, -1:], Dk - T, 1)], 1)).swapaxes(1, 2)[..., None]
    out = np.exp(G - np.where((t % 2 == 0)[None, :, None], G[:, t // 2], 0.0))[..., None]
    live = n > 0
    units = 2.5 * 2.0 ** -23
    # some of the sums pass -87.3, where the exponential is below 2^-126, the smallest normal number: the hardware gives 0 for
    # it, which is off by less than 2^-126 (and so is a part below it that counts as 0)
    least = 2.0 ** -126
    off = np.abs(final[live] - want[live]) - least
    assert (off <= units * want[live]).all(), (off / want[live]).max() * 2 ** 23
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    off = np.abs(o[live] - out[live]) - least
    assert (off <= (units + half) * out[live]).all(), (off / out[live]).max() * 2 ** 23
