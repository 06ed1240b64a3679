"""The forms of the operators around the scan on the CPU: which calls take which form, the forms that only
larger calls take at sizes that the emulator can run, and the order in which waves run."""

import ctypes
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import operators_cases as cases
import operators_form_cases as forms
import operators_ref as ref
import ops_emu_harness as harness
from test_operators_edges import _Run, library  # noqa: F401


@pytest.fixture(scope="module")
def lib(library):  # noqa: F811
    loaded = harness.load(library)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    loaded.emu_fp8_form.argtypes = [i64, i64, i64, i32, i32, vp]
    loaded.emu_gated_form.argtypes = [i64, i64, i64, i32, i32, vp]
    loaded.emu_fp8_form.restype = loaded.emu_gated_form.restype = None
    loaded.emu_fp8_big.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    return loaded


def _fp8_form(lib, M, N, K, out):
    f = (ctypes.c_int64 * 5)()
    lib.emu_fp8_form(M, N, K, harness.KIND[out], K % 16 == 0, f)
    return ("few", f[1], f[2]) if f[0] else ("big", f[1], f[3] > 1)


def test_the_calls_of_the_gpu_tests_take_every_form(lib):
    seen = set()
    for M, N, K, out, form in forms.MATMUL:
        assert _fp8_form(lib, M, N, K, out) == form, (M, N, K, out)
        seen.add(form + (out,))
    assert seen == forms.MATMUL_FORMS
    forwards, backwards = set(), set()
    for B, T, C, kind, forward, backward in forms.GATED:
        for want, back, all_of in ((forward, 0, forwards), (backward, 1, backwards)):
            f = (ctypes.c_int64 * 3)()
            lib.emu_gated_form(B, T, C, harness.KIND[kind], back, f)
            assert (f[0], f[1] > 1, bool(f[2])) == want, (B, T, C, kind, back)
            all_of.add(want + (kind,))
    assert forwards == forms.GATED_FORMS | forms.GATED_WALKS and backwards == forms.GATED_FORMS


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K,out", [(5, 40, 1300, "bf16"), (20, 33, 2100, "f32"), (31, 17, 1160, "bf16"), (40, 20, 1200, "f32")])
def test_few_rows_and_a_long_sum(lib, M, N, K, out, block_rows):
    """The few-row product with 8 and 16 waves."""
    assert _fp8_form(lib, M, N, K, out)[2] > 4
    cases.matmul(_Run(lib), M, N, K, block_rows, out, 0, 0, 3)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K,splits", [(300, 270, 400, 1), (257, 513, 128, 1), (260, 100, 1040, 3), (1, 1, 16, 1)])
def test_large_tiles(lib, M, N, K, splits, block_rows):
    """The product in tiles of 256 x 256."""
    a, sa, b, sb = cases.matmul_inputs(M, N, K, block_rows, M + K)
    want, err = ref.matmul(ref.E4M3[a], sa, ref.E4M3[b], sb, block_rows, "bf16")
    A, B = (harness.Guarded(v.size, 16).write(v.tobytes()) for v in (a, b))
    SA, SB = harness.put(sa, "f32"), harness.put(sb, "f32")
    out, part = harness.Guarded(2 * M * N, 2), harness.Guarded(4 * splits * M * N, 4)
    assert lib.emu_fp8_big(A.at, SA.at, B.at, SB.at, M, N, K, block_rows, splits, out.at, part.at) == 0
    ref.close(harness.get(out, "bf16", (M, N)), want, err, "bf16", "out")


def test_rows_beyond_the_workgroups(lib):
    """A norm whose workgroups of four waves each walk over two rows."""
    cases.norm(_Run(lib), 2051, 1030, "f32", True, 0)
    cases.norm_backward(_Run(lib), 1027, 1030, "bf16", True, 0)


def test_shuffled_waves_give_the_same_bits(lib):
    """A missing barrier would make results depend on the order in which waves run: segments and their
    folds, products of few rows and of split sums, norms that meet in shared memory over two rows."""
    run = _Run(lib)
    x, gi, gr, lam, init, n = ref.gated_case(1, 1100, 70, "f32", 3, state=True, lengths=[1050])
    y, yi, yr, ylam, _, _ = ref.gated_case(1, 800, 132, "bf16", 4)
    gh = np.random.default_rng(2).standard_normal(x.shape)
    states = ref.gated(x, gi, gr, lam, 8.0, init, n)[0][2]
    few, wide, long = (cases.matmul_inputs(M, N, K, 1, M) for M, N, K in ((20, 33, 1300), (70, 90, 400), (70, 40, 3000)))
    _, nx, nres, nw = cases.norm_inputs(2050, 1030, "bf16", True, 1)
    seen = []
    for seed in (0, 1, 12345):
        lib.emu_set_shuffle_seed(seed)
        out = [run.gated(x, gi, gr, lam, 8.0, "f32", init=init, lengths=n, states=True),
               run.gated_backward(x, gi, gr, lam, 8.0, "f32", states, gh, gfinal=init, lengths=n),
               run.gated(y, yi, yr, ylam, 8.0, "bf16", states=True)]
        out += [[run.matmul(*m, 1, out) for out in ("bf16", "f32")] for m in (few, wide, long)]
        out += [[v for v in run.norm(nx, nres, nw, 1e-6, "bf16").values()],
                run.norm_backward(nx[:1026], nw, np.ones(1026), nres[:1026], None, "bf16")]
        seen.append([np.asarray(v) for group in out for v in group])
    lib.emu_set_shuffle_seed(0)
    for s in seen[1:]:
        assert [k for k, (v, w) in enumerate(zip(seen[0], s)) if not np.array_equal(v, w)] == []
