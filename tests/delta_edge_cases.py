"""Further cases of the gated delta rule that the emulator and the GPU run alike (test-only), as delta_cases: each takes a
`run` with the functions of delta_emu_harness."""

import numpy as np

import delta_cases
import delta_ref as ref

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


def _two(rows, longest, other):
    """Lengths of many rows, all but two of them empty."""
    n = [0] * rows
    n[rows // 2], n[-1] = longest, other
    return n


# As delta_cases.DELTA, with so many heads that the walks make their triangles themselves: with up to 64 and up to 128 features,
# by 64 and by 128 columns to a workgroup. Sizes that are no multiple of four, columns that end inside a wave and inside a
# workgroup, rows of tokens apart, tokens that forget, poisoned padding, rows without tokens.
MANY = [
    (97, 200, 1, 2, 33, 21, "f32", True, _two(97, 200, 131), 3, True),
    (97, 200, 2, 2, 64, 64, "bf16", False, _two(97, 199, 64), 0, True),
    (97, 130, 1, 2, 17, 50, "bf16", True, _two(97, 130, 65), 5, False),
    (97, 130, 2, 2, 72, 48, "bf16", True, _two(97, 129, 1), 0, True),
    (97, 130, 1, 2, 100, 33, "f32", True, _two(97, 130, 70), 1, False),
    (97, 130, 1, 2, 128, 64, "f32", True, _two(97, 128, 63), 0, False),
    (97, 130, 1, 1, 66, 70, "f32", True, _two(97, 130, 66), 7, True),
    (97, 130, 1, 1, 128, 128, "bf16", False, _two(97, 130, 127), 0, False),
    (65, 130, 1, 1, 50, 255, "bf16", True, _two(65, 130, 100), 2, False),
    (65, 130, 1, 1, 128, 255, "f32", True, _two(65, 130, 96), 0, True),
    (65, 70, 1, 1, 127, 130, "bf16", True, _two(65, 70, 9), 1, False),
    (97, 9, 2, 2, 64, 64, "bf16", True, _two(97, 9, 5), 0, False),
]


def shuffled(run, shuffle):
    """Two cases of many heads under several orders of their waves: the same bits."""
    for sizes, seed in (((97, 140, 1, 2, 40, 50, "bf16"), 9), ((97, 140, 1, 1, 70, 66, "f32"), 10)):
        kind = sizes[-1]
        q, k, v, g, beta, init, n = ref.case(*sizes, seed, lengths=_two(sizes[0], 140, 65))
        states = np.float32(ref.tokens(q, k, v, g, beta, 1.0, init, n)[2])
        got = []
        for order in (0, 1, 12345, 987654321):
            shuffle(order)
            got.append(list(run.delta(q, k, v, g, beta, 1.0, kind, init=init, lengths=n, states=True))
                       + run.delta_backward(q, k, v, g, beta, 1.0, kind, states, v, gfinal=init, lengths=n))
        shuffle(0)
        assert all(np.array_equal(a, b) for o in got[1:] for a, b in zip(o, got[0]))


def _padded(x, rows):
    """x's rows in front of many empty ones."""
    return None if x is None else np.concatenate([x] + [np.zeros((rows - len(x),) + x.shape[1:])])


class InABatch:
    """A run whose calls have their rows in front of many that hold no tokens, so that the walks over many heads take them."""

    def __init__(self, run, rows):
        self._run, self._rows = run, rows

    def _lengths(self, v, lengths):
        n = np.full(v.shape[0], v.shape[1]) if lengths is None else np.asarray(lengths)
        return np.concatenate([n, np.zeros(self._rows - len(n))]).astype(np.int32)

    def delta(self, q, k, v, g, beta, scale, kind, init=None, lengths=None, **more):
        wide = [_padded(w, self._rows) for w in (q, k, v, g, beta)]
        got = self._run.delta(*wide, scale, kind, init=_padded(init, self._rows), lengths=self._lengths(v, lengths), **more)
        return tuple(None if w is None else w[:len(v)] for w in got)

    def delta_backward(self, q, k, v, g, beta, scale, kind, states, go, gfinal=None, lengths=None, **more):
        wide = [_padded(w, self._rows) for w in (q, k, v, g, beta)]
        got = self._run.delta_backward(*wide, scale, kind, _padded(states, self._rows), _padded(go, self._rows),
                                       gfinal=_padded(gfinal, self._rows), lengths=self._lengths(v, lengths), **more)
        return [w[:len(v)] for w in got]


def many(run):
    """(name, function): what delta_cases holds the walks over few heads to, of those over many."""
    batch = InABatch(run, 193)
    todo = [("%s %s" % (f.__name__, kind), lambda f=f, kind=kind: f(batch, kind)) for f in (delta_cases.same_keys, delta_cases.columns_apart)
            for kind in ("f32", "bf16")]
    return todo + [("clamped", lambda: delta_cases.clamped(batch)), ("empty row", lambda: delta_cases.empty_row_infinite(batch))]


def outputs(run, B, T, Hk, Hv, Dk, Dv, kind, state, lengths, pad, forget):
    """bfloat16 outputs within the bounds of products in 24 bits, and their own rounding."""
    q, k, v, g, beta, init, n = ref.case(B, T, Hk, Hv, Dk, Dv, kind, B * 1000 + T + Dv + 7, state, lengths, forget)
    want = ref.forward(q, k, v, g, beta, 0.9, init, n, "f32")
    ref.close(run.delta(q, k, v, g, beta, 0.9, kind, init=init, lengths=n, pad=pad)[0], want[0], kind, "o")


OUTPUTS = [c for c in delta_cases.DELTA + MANY if c[6] == "bf16"]
