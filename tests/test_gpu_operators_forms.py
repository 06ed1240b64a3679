"""Every form of the operators around the scan on the GPU: the calls of operators_form_cases, whose forms
test_operators_forms checks against the plans, each against float64."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import complex_chunkwise_ssd_amd as ssd
import operators_cases as cases
import operators_form_cases as forms
import operators_ref as ref
from test_gpu_operators import _Gpu

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
FP8 = torch.float8_e4m3fn


def _spread(scale, block_rows, R, K):
    """The scale of every value, float64 (R, K)."""
    s = scale.double()
    s = s.t() if block_rows == 1 else s.repeat_interleave(128, 0)[:R]
    return s.repeat_interleave(128, 1)[:, :K]


def _groups_top(v):
    """The largest magnitude of each eight neighbouring k (R, ceil(K / 8))."""
    v = torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 8))
    return v.reshape(v.shape[0], -1, 8).amax(2)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K,out,form", forms.MATMUL, ids=str)
def test_fp8_matmul(M, N, K, out, form, block_rows):
    """operators_ref.matmul's bound; the largest product of a group of eight is at most the product of the
    operands' largest. Rows of K a multiple of 16 as they lie, others laid out anew."""
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    a, b = (torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8) for s in ((M, K), (N, K)))
    for v in (a, b):
        v[(v & 127) == 127] ^= 1      # no NaN
    kb = -(-K // 128)
    sa = torch.exp(torch.randn(kb, M, generator=g, device=DEV))
    sb = torch.exp(torch.randn(*((kb, N) if block_rows == 1 else (-(-N // 128), kb)), generator=g, device=DEV))
    got = ssd.fp8_matmul(a.view(FP8), sa, b.view(FP8), sb, block_rows=block_rows,
                         out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    av = a.view(FP8).double() * _spread(sa, 1, M, K)
    bv = b.view(FP8).double() * _spread(sb, block_rows, N, K)
    want = av @ bv.t().contiguous()
    err = ref.U * (2 * 64 + 4 + 2 * kb) * (av.abs() @ bv.abs().t().contiguous())
    if out == "bf16":
        err += 7 * 2.0 ** -13 * (_groups_top(av) @ _groups_top(bv).t().contiguous())
    bar = err + ref.HALF[out] * (want.abs() + err)
    off = (got.double() - want).abs()
    assert torch.isfinite(off).all()
    bad = off > bar
    assert not bad.any(), "%d off, worst %.3g of its bar at %s" % (bad.sum(), (off / bar).max(), bad.nonzero()[0])
    again = ssd.fp8_matmul(a.view(FP8), sa, b.view(FP8), sb, block_rows=block_rows, out_dtype=got.dtype)
    assert torch.equal(got, again)


@pytest.mark.parametrize("B,T,C,kind,forwards,backwards", forms.GATED, ids=str)
def test_gated_scan(B, T, C, kind, forwards, backwards):
    lengths = [T - (T // 2) * (b % 3 == 1) for b in range(B)]
    cases.gated(_Gpu, B, T, C, kind, True, lengths, 2)
    cases.gated_backward(_Gpu, B, T, C, kind, True, lengths, 2)


@pytest.mark.parametrize("rows,F,kind", forms.NORM, ids=str)
def test_rms_norm(rows, F, kind):
    cases.norm(_Gpu, rows, F, kind, True, 0)
    cases.norm_backward(_Gpu, rows, F, kind, True, 0)
