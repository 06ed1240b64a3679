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


ALL = {f.__name__: f for f in (gated_lengths_lowest,)}
