"""The norms around a block on the CPU: the unchanged kernel and C-ABI sources under the host wave emulator,
against float64 formulas. The whole set runs in one process of its own (this file run as a program): every
buffer ends at a page that cannot be touched."""

import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import block_norm_cases as cases
import block_norm_harness as harness


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
        todo.append(("gated %s" % (c,), lambda c=c: cases.run_gated(run, *c)))
        todo.append(("gated backward %s" % (c,), lambda c=c: cases.run_gated_backward(run, *c)))
    for c in cases.BLOCK:
        todo.append(("block %s" % (c,), lambda c=c: cases.run_block(run, *c)))
        todo.append(("block backward %s" % (c,), lambda c=c: cases.run_block_backward(run, *c)))
    todo.append(("rows apart", lambda: cases.rows_apart(run)))
    return todo


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    lib = harness.build(str(tmp_path_factory.mktemp("block_emu")))
    return subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True, text=True)


def test_every_case(report):
    assert report.returncode == 0 and report.stdout.rstrip().endswith("all done"), \
        report.stdout[-2000:] + report.stderr[-2000:]


def test_shuffled_waves_give_the_same_bits(report):
    # a missing barrier would make results depend on the order in which waves run
    assert "shuffled: the same" in report.stdout, report.stdout[-2000:] + report.stderr[-2000:]


def _differences(loss, args, want, seed):
    r = np.random.default_rng(seed)
    for i, w in enumerate(want):
        for at in [tuple(r.integers(0, s) for s in w.shape) for _ in range(8)]:
            up, down = [[a.copy() for a in args] for _ in range(2)]
            up[i][at] += 1e-5
            down[i][at] -= 1e-5
            d = (loss(*up) - loss(*down)) / 2e-5
            assert abs(d - w[at]) < 1e-7 * (1 + abs(d)), (i, at, d, w[at])


def test_gradient_formulas_agree_with_differences():
    """The float64 gradients that the kernels are held to, against central differences."""
    g = np.random.default_rng(3)
    x, z, gy, gs = (g.standard_normal((4, 20)) for _ in range(4))
    w = 1 + 0.2 * g.standard_normal(10)
    rstd = cases.gated(x, z, w, 10, 1e-6)[0][1]
    _differences(lambda x, z, w: (gy * cases.gated(x, z, w, 10, 1e-6)[0][0]).sum(), [x, z, w],
                 cases.gated_backward(x, z, w, rstd, gy)[0], 1)
    w1, w2 = 1 + 0.2 * g.standard_normal(20), 1 + 0.2 * g.standard_normal(20)
    (_, s, r1, r2), _ = cases.block(x, z, w1, w2, 0.4, 1e-6)

    def loss(x, res, w1, w2):
        y, s = cases.block(x, res, w1, w2, 0.4, 1e-6)[0][:2]
        return (gy * y).sum() + (gs * s).sum()

    _differences(loss, [x, z, w1, w2], cases.block_backward(x, s, w1, w2, r1, r2, 0.4, gy, gs)[0], 2)


def _shuffled(lib):
    """Some cases under several thread orders: the same bits."""
    run, got = _Run(lib), []
    g = np.random.default_rng(9)
    for seed in (0, 1, 12345, 987654321):
        lib.emu_set_shuffle_seed(seed)
        g = np.random.default_rng(9)
        out = []
        for rows, H, D in ((9, 3, 43), (3, 17, 120), (20, 2, 16)):
            x, z, gy = (g.standard_normal((rows, H * D)) for _ in range(3))
            w, w2 = g.standard_normal(D), g.standard_normal(H * D)
            f = run.gated_norm(x, z, w, 1e-6, "bf16")
            out += [*f.values(), *run.gated_norm_backward(x, z, w, f["rstd"], gy, "bf16")]
            b = run.block_norm(x, z, w2, w2, 0.5, 1e-6, "bf16", in_place=True)
            out += [*b.values(), *run.block_norm_backward(x, z, w2, w2, b["post"], b["pre"], 0.5, gy, gy, "bf16")]
        got.append(out)
    lib.emu_set_shuffle_seed(0)
    return all(np.array_equal(a, b) for o in got[1:] for a, b in zip(o, got[0]))


if __name__ == "__main__":
    loaded = harness.load(sys.argv[1])
    for name, fn in everything(loaded):
        print(name, flush=True)
        fn()
    print("shuffled: the same" if _shuffled(loaded) else "shuffled: DIFFERENT", flush=True)
    print("all done", flush=True)
