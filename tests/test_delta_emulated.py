"""The gated delta rule on the CPU: the unchanged kernel and C-ABI sources under the host wave emulator,
against float64 formulas. The whole set runs in one process of its own (this file run as a program): every
buffer ends at a page that cannot be touched."""

import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import delta_cases as cases
import delta_emu_harness as harness
import delta_ref as ref


class _Run:
    """The harness bound to a library."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        return lambda *a, **k: getattr(harness, name)(self._lib, *a, **k)


def everything(lib):
    """(name, function) of every case."""
    run = _Run(lib)
    todo = []
    for c in cases.DELTA:
        todo.append(("forward %s" % (c,), lambda c=c: cases.forward(run, *c)))
        todo.append(("backward %s" % (c,), lambda c=c: cases.backward(run, *c)))
    for kind in ("f32", "bf16"):
        todo.append(("same keys %s" % kind, lambda kind=kind: cases.same_keys(run, kind)))
        todo.append(("columns apart %s" % kind, lambda kind=kind: cases.columns_apart(run, kind)))
    todo.append(("clamped", lambda: cases.clamped(run)))
    todo.append(("empty row, infinite gradient", lambda: cases.empty_row_infinite(run)))
    return todo


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    lib = harness.build(str(tmp_path_factory.mktemp("delta_emu")))
    return subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True, text=True)


def test_every_case(report):
    assert report.returncode == 0 and report.stdout.rstrip().endswith("all done"), \
        report.stdout[-2000:] + report.stderr[-2000:]


def test_shuffled_waves_give_the_same_bits(report):
    # a missing barrier would make results depend on the order in which waves run
    assert "shuffled: the same" in report.stdout, report.stdout[-2000:] + report.stderr[-2000:]


def test_the_bounds_hold_the_definition():
    """The chunked form that the bounds are made for against the definition, one token after the other."""
    q, k, v, g, beta, init, n = ref.case(2, 150, 1, 2, 12, 10, "f32", 4, lengths=[150, 70], forget=True)
    got = ref.forward(q, k, v, g, beta, 0.3, init, n, "f32")
    for x, y in zip(got, ref.tokens(q, k, v, g, beta, 0.3, init, n)):
        assert np.abs(x.v - y).max() < 1e-12
    r = np.random.default_rng(2)
    go, gf = r.standard_normal(v.shape), r.standard_normal(init.shape)
    got = ref.backward(q, k, v, g, beta, 0.3, ref.tokens(q, k, v, g, beta, 0.3, init, n)[2], go, gf, n)
    for x, y in zip(got, ref.tokens_backward(q, k, v, g, beta, 0.3, init, go, gf, n)):
        assert np.abs(x.v - y).max() < 1e-11


def test_gradient_formulas_agree_with_differences():
    """The float64 gradients that the kernels are held to, against central differences."""
    q, k, v, g, beta, init, n = ref.case(2, 9, 1, 2, 4, 3, "f32", 5, lengths=[9, 4])
    r = np.random.default_rng(1)
    go, gf = r.standard_normal(v.shape), r.standard_normal(init.shape)

    def loss(q, k, v, g, beta, init):
        o, final, _ = ref.tokens(q, k, v, g, beta, 0.4, init, n)
        return (go * o).sum() + (gf * final).sum()

    args = [q, k, v, g, beta, init]
    want = ref.tokens_backward(q, k, v, g, beta, 0.4, init, go, gf, n)
    for i, w in enumerate(want):
        for at in [tuple(r.integers(0, s) for s in w.shape) for _ in range(12)]:
            e = 1e-5
            up, down = [[a.copy() for a in args] for _ in range(2)]
            up[i][at] += e
            down[i][at] -= e
            d = (loss(*up) - loss(*down)) / (2 * e)
            assert abs(d - w[at]) < 1e-7 * (1 + abs(d)), (i, at, d, w[at])


def _shuffled(lib):
    """Two cases under several thread orders: the same bits."""
    run = _Run(lib)
    q, k, v, g, beta, init, n = ref.case(2, 140, 1, 2, 40, 70, "bf16", 9, lengths=[140, 65])
    states = np.float32(ref.tokens(q, k, v, g, beta, 1.0, init, n)[2])
    got = []
    for seed in (0, 1, 12345, 987654321):
        lib.emu_set_shuffle_seed(seed)
        got.append(list(run.delta(q, k, v, g, beta, 1.0, "bf16", init=init, lengths=n, states=True))
                   + run.delta_backward(q, k, v, g, beta, 1.0, "bf16", states, v, gfinal=init, lengths=n))
    lib.emu_set_shuffle_seed(0)
    return all(np.array_equal(a, b) for o in got[1:] for a, b in zip(o, got[0]))


if __name__ == "__main__":
    loaded = harness.load(sys.argv[1])
    for name, fn in everything(loaded):
        print(name, flush=True)
        fn()
    print("shuffled: the same" if _shuffled(loaded) else "shuffled: DIFFERENT", flush=True)
    print("all done", flush=True)
