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
