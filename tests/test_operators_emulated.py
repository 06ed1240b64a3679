"""The operators around the scan on the CPU: the unchanged kernel and C-ABI sources under the
host wave emulator, against float64 formulas. Every buffer ends at a page that cannot be
touched. The whole set runs in one process of its own (this file run as a program), so that
such an access ends that process and not the test run."""

import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import operators_cases as cases
import operators_ref as ref
import ops_emu_harness as harness


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
    for c in cases.GATED:
        todo.append(("gated %s" % (c,), lambda c=c: cases.gated(run, *c)))
        todo.append(("gated_backward %s" % (c,), lambda c=c: cases.gated_backward(run, *c)))
    for c in cases.NORM:
        todo.append(("norm %s" % (c,), lambda c=c: cases.norm(run, *c)))
        todo.append(("norm_backward %s" % (c,), lambda c=c: cases.norm_backward(run, *c)))
    for b in (1, 128):
        for turn in (False, True):
            for c in cases.QUANTISE:
                todo.append(("quantise %s %s %s" % (c, b, turn), lambda c=c, b=b, turn=turn: cases.quantise(run, *c, b, turn)))
            todo.append(("quantise_special %s %s" % (b, turn), lambda b=b, turn=turn: cases.quantise_special(run, b, turn)))
    for c in cases.MATMUL:
        for align in (16, 1):
            todo.append(("matmul %s align %d" % (c, align), lambda c=c, align=align: cases.matmul(run, *c, align=align)))
    todo.append(("gated lengths clamped", lambda: cases.gated_lengths_clamped(run)))
    todo.append(("gated empty row, infinite gradient", lambda: cases.gated_empty_row_infinite(run)))
    for M in (5, 70):
        for out in ("bf16", "f32"):
            todo.append(("matmul_special %d %s" % (M, out), lambda M=M, out=out: cases.matmul_special(run, M, out)))
    return todo


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    lib = harness.build(str(tmp_path_factory.mktemp("ops_emu")))
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True, text=True)
    return r


def test_every_case(report):
    assert report.returncode == 0 and report.stdout.rstrip().endswith("all done"), \
        report.stdout[-2000:] + report.stderr[-2000:]


def test_shuffled_waves_give_the_same_bits(report):
    # a missing barrier would make results depend on the order in which waves run
    assert "shuffled: the same" in report.stdout, report.stdout[-2000:] + report.stderr[-2000:]


def test_gradient_formulas_agree_with_differences():
    """The float64 gradients that the kernels are held to, against central differences."""
    x, gi, gr, lam, init, n = ref.gated_case(2, 9, 3, "f32", 5, state=True, lengths=[9, 4])
    g = np.random.default_rng(1)
    gh, gf = g.standard_normal((2, 9, 3)), g.standard_normal((2, 3))

    def loss(*v):
        h, final, _ = ref.gated(*v[:4], 8.0, v[4], n)[0]
        return (h * gh).sum() + (final * gf).sum()
    args = [x, gi, gr, lam, init]
    got = ref.gated_backward(x, gi, gr, lam, 8.0, init, gh, gf, n)[0]
    for k in range(5):
        for at in np.ndindex(args[k].shape):
            d, pair = 1e-5, []
            for sign in (1, -1):
                v = [a.copy() for a in args]
                v[k][at] += sign * d
                pair.append(loss(*v))
            # a central difference is off by d^2 times the third derivative: 1e-10 of O(1) values
            assert abs((pair[0] - pair[1]) / (2 * d) - got[k][at]) <= 1e-6 * (1 + abs(got[k][at])), (k, at)
    s, w = g.standard_normal((3, 5)), g.standard_normal(5)
    gy, gs = g.standard_normal((3, 5)), g.standard_normal((3, 5))

    def norm_loss(s, w):
        (y, _, _), _ = ref.norm(s, None, w, 1e-6)
        return (y * gy).sum() + (s * gs).sum()
    rstd = 1 / np.sqrt((s * s).mean(1) + 1e-6)
    (gx, gw), _ = ref.norm_backward(s, w, rstd, gy, gs)
    for v, grad, k in ((s, gx, 0), (w, gw, 1)):
        for at in np.ndindex(v.shape):
            pair = []
            for sign in (1, -1):
                u = v.copy()
                u[at] += sign * 1e-5
                pair.append(norm_loss(u, w) if k == 0 else norm_loss(s, u))
            assert abs((pair[0] - pair[1]) / 2e-5 - grad[at]) <= 1e-6 * (1 + abs(grad[at]))


if __name__ == "__main__":
    library = harness.load(sys.argv[1])
    only = sys.argv[2:]
    for name, fn in everything(library):
        if only and not any(o in name for o in only):
            continue
        print(name, flush=True)
        fn()
    run = _Run(library)
    x, gi, gr, lam, init, _ = ref.gated_case(1, 300, 70, "f32", 3, state=True)
    gh = np.random.default_rng(2).standard_normal(x.shape)
    states = ref.gated(x, gi, gr, lam, 8.0, init)[0][2]
    a, sa, b, sb = cases.matmul_inputs(70, 90, 400, 128, 1)
    _, nx, nres, nw = cases.norm_inputs(3, 3000, "bf16", True, 1)
    seen = []
    for seed in (0, 1, 12345):
        library.emu_set_shuffle_seed(seed)
        out = [run.gated(x, gi, gr, lam, 8.0, "f32", init=init)[:2],
               run.gated_backward(x, gi, gr, lam, 8.0, "f32", states, gh),
               [run.matmul(a, sa, b, sb, 128, "f32")],
               [v for v in run.norm(nx, nres, nw, 1e-6, "bf16").values()],
               run.norm_backward(nx, nw, np.ones(3), nres, None, "bf16"),
               run.quantise(nx, "bf16", 1, True), run.quantise(nx, "bf16", 128, True)]
        seen.append([np.asarray(v) for group in out for v in group])
    library.emu_set_shuffle_seed(0)
    same = all(np.array_equal(v, w) for s in seen[1:] for v, w in zip(seen[0], s))
    print("shuffled: %s" % ("the same" if same else "DIFFERENT"))
    print("all done")
