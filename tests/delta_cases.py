"""Cases of the gated delta rule that the emulator and the GPU run alike (test-only). Each takes a `run`
with the functions of delta_emu_harness (numpy in, numpy out)."""

import numpy as np

import delta_ref as ref

NAN = float("nan")

# B, T, Hk, Hv, Dk, Dv, kind, state, lengths, padding between tokens, tokens that forget
DELTA = [
    (1, 1, 1, 1, 1, 1, "f32", True, None, 0, False),
    (2, 1, 2, 4, 64, 64, "bf16", True, [1, 0], 3, False),
    (1, 5, 1, 2, 72, 100, "bf16", True, None, 0, True),
    (3, 8, 1, 1, 128, 66, "f32", True, [8, 3, 0], 1, False),
    (1, 3, 2, 2, 17, 5, "bf16", False, None, 2, False),
    (2, 9, 1, 1, 16, 16, "f32", True, [9, 4], 0, False),
    (1, 63, 1, 2, 64, 64, "bf16", False, None, 0, False),
    (1, 64, 1, 1, 33, 65, "f32", True, None, 5, True),
    (2, 65, 1, 1, 64, 48, "bf16", True, [65, 64], 0, False),
    (1, 150, 1, 3, 40, 20, "f32", False, None, 0, False),
    (2, 130, 1, 2, 100, 72, "bf16", True, [129, 33], 7, True),
    (1, 200, 1, 1, 128, 130, "f32", True, [140], 0, False),
    (3, 70, 1, 1, 7, 9, "bf16", True, [0, 1, 70], 1, False),
    (1, 100, 1, 1, 128, 256, "bf16", True, None, 0, False),
]


def _poisoned(n, T, *arrays):
    if n is None:
        return arrays
    dead = np.arange(T)[None, :] >= n[:, None]
    out = []
    for i, w in enumerate(arrays):
        out.append(np.where(dead.reshape(dead.shape + (1,) * (w.ndim - 2)), (NAN, np.inf, -np.inf)[i % 3], w))
    return out


def forward(run, B, T, Hk, Hv, Dk, Dv, kind, state, lengths, pad, forget):
    q, k, v, g, beta, init, n = ref.case(B, T, Hk, Hv, Dk, Dv, kind, B * 1000 + T + Dk, state, lengths, forget)
    scale = Dk ** -0.5
    want = ref.forward(q, k, v, g, beta, scale, init, n, kind)
    q, k, v, g, beta = _poisoned(n, T, q, k, v, g, beta)
    o, final, states = run.delta(q, k, v, g, beta, scale, kind, init=init, lengths=n, states=True, pad=pad)
    ref.close(o, want[0], kind, "o")
    ref.close(final, want[1], "f32", "final")
    ref.close(states, want[2], "f32", "states")
    if init is not None:
        again = run.delta(q, k, v, g, beta, scale, kind, init=init, lengths=n, pad=pad, in_place=True)
        assert np.array_equal(again[0], o) and np.array_equal(again[1], final)


def backward(run, B, T, Hk, Hv, Dk, Dv, kind, state, lengths, pad, forget):
    q, k, v, g, beta, init, n = ref.case(B, T, Hk, Hv, Dk, Dv, kind, B * 1000 + T + Dv, True, lengths, forget)
    scale = 0.7
    r = np.random.default_rng(T)
    go = ref.rounded(r.standard_normal(v.shape), kind)
    gf = np.float32(r.standard_normal(init.shape)).astype(np.float64) if state else None
    states = np.float32(ref.tokens(q, k, v, g, beta, scale, init, n)[2]).astype(np.float64)
    want = ref.backward(q, k, v, g, beta, scale, states, go, gf, n)
    q, k, v, g, beta, go = _poisoned(n, T, q, k, v, g, beta, go)
    got = run.delta_backward(q, k, v, g, beta, scale, kind, states, go, gfinal=gf, lengths=n, pad=pad)
    for name, x, w, t in zip(("q", "k", "v", "g", "beta", "init"), got, want, (kind, kind, kind, "f32", "f32", "f32")):
        ref.close(x, w, t, "grad " + name)


def same_keys(run, kind, n=None):
    """Every key the same and no decay: the system that is solved has ones all below its diagonal times
    beta, where powers of it grow without bound. And strengths of 0, 1 and 2."""
    B, T, Dk, Dv = 1, 130, 20, 24
    q, k, v, _, _, init, _ = ref.case(B, T, 1, 1, Dk, Dv, kind, 3)
    k = np.broadcast_to(ref.rounded(np.eye(Dk)[3], kind), k.shape).copy()
    g = np.zeros((B, T, 1))
    for beta in (np.ones((B, T, 1)), np.full((B, T, 1), 2.0), np.zeros((B, T, 1)),
                 np.arange(T).reshape(B, T, 1) % 3 * 1.0):
        o, final, states = ref.tokens(q, k, v, g, beta, 1.0, init)
        got = run.delta(q, k, v, g, beta, 1.0, kind, init=init)
        # every number here is a sum of at most T values of v and the state, each exact in the parts: the
        # alternating sums that beta = 2 makes of them have up to T terms, rounded T times
        bar = ref.U * 4 * T * (T + 64)
        assert np.abs(got[1] - final).max() <= bar
        assert (np.abs(got[0] - o) <= bar + ref.HALF[kind] * (np.abs(o) + bar) + 2.0 ** -15 * np.abs(q).sum(-1, keepdims=True)
                * (T + 8) * (kind == "bf16")).all()


def clamped(run):
    """Lengths below 0 and past T count as 0 and T; a decay of minus infinity forgets."""
    q, k, v, g, beta, init, _ = ref.case(3, 70, 1, 1, 12, 10, "f32", 5)
    g[:, 40] = -np.inf
    a = run.delta(q, k, v, g, beta, 1.0, "f32", init=init, lengths=np.array([-3, 75, 2 ** 31 - 1], np.int32))
    b = run.delta(q, k, v, g, beta, 1.0, "f32", init=init, lengths=np.array([0, 70, 70], np.int32))
    assert all(np.array_equal(x, y) for x, y in zip(a[:2], b[:2]))
    g[:, 40] = -1000.0
    want = ref.forward(q, k, v, g, beta, 1.0, init, np.array([0, 70, 70]), "f32")
    ref.close(a[0], want[0], "f32", "o")
    ref.close(a[1], want[1], "f32", "final")
    few = slice(0, 3)
    g[:, 1] = -np.inf
    c = run.delta(*(w[:, few] for w in (q, k, v, g, beta)), 1.0, "f32", init=init)
    g[:, 1] = -1000.0
    want = ref.forward(*(w[:, few] for w in (q, k, v, g, beta)), 1.0, init, None, "f32")
    ref.close(c[0], want[0], "f32", "o")


def columns_apart(run, kind):
    """A NaN or an infinity in a column of v stays in that column of its head; one in q stays with its
    token."""
    q, k, v, g, beta, init, _ = ref.case(1, 70, 1, 2, 24, 20, kind, 6)
    clean = run.delta(q, k, v, g, beta, 1.0, kind, init=init)
    for bad in (NAN, np.inf):
        w = v.copy()
        w[0, 66, 0, 3] = bad
        o, final, _ = run.delta(q, k, w, g, beta, 1.0, kind, init=init)
        assert not np.isfinite(final[0, 0, :, 3]).any() and not np.isfinite(o[0, 66:, 0, 3]).any()
        o[0, 64:, 0, 3], final[0, 0, :, 3] = clean[0][0, 64:, 0, 3], clean[1][0, 0, :, 3]
        assert np.array_equal(o, clean[0]) and np.array_equal(final, clean[1])
        w = q.copy()
        w[0, 5, 0, 2] = bad
        o, final, _ = run.delta(w, k, v, g, beta, 1.0, kind, init=init)
        assert not np.isfinite(o[0, 5]).any()
        o[0, 5] = clean[0][0, 5]
        assert np.array_equal(o, clean[0]) and np.array_equal(final, clean[1])


def empty_row_infinite(run):
    """A row without tokens hands its final state's gradient on and leaves the others' alone, be it
    infinite."""
    q, k, v, g, beta, init, _ = ref.case(2, 70, 1, 1, 12, 10, "f32", 8)
    n = np.array([70, 0], np.int32)
    states = ref.tokens(q, k, v, g, beta, 1.0, init, n)[2]
    gf = np.ones(init.shape)
    want = run.delta_backward(q, k, v, g, beta, 1.0, "f32", states, v, gfinal=gf, lengths=n)
    gf[1] = np.inf
    got = run.delta_backward(q, k, v, g, beta, 1.0, "f32", states, v, gfinal=gf, lengths=n)
    assert all(np.array_equal(a, b) for a, b in zip(got[:5], want[:5]))
    assert np.array_equal(got[5][0], want[5][0]) and np.isposinf(got[5][1]).all()
