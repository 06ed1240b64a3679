"""The weights' gradients of the norms around a block over very many rows: a lane adds at most 256 of them in float32, what is
added further is float64, so that errors do not grow with the rows."""

import os

import pytest
import torch

import complex_chunkwise_ssd_amd as ssd

U = 2.0 ** -24
CHAIN = 256


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(ssd.LIBPATH):
        from complex_chunkwise_ssd_amd import build
        build.build()


def _held(F):
    """Rows that a workgroup holds at once."""
    return 16 if F <= 128 else 4 if F <= 1024 else 1


@pytest.mark.parametrize("F", [8, 128, 129, 1024, 1025, 4096, 4097, 16384])
def test_shares_grow_with_the_rows(F):
    for rows in (1, 5000, 1 << 20, 1 << 23, (1 << 26) + 3):
        groups = ssd.block.block_norm_backward_workspace_bytes(rows, F) / (8 * F)
        assert groups * _held(F) * CHAIN >= rows, rows
        if F >= 64:  # the heads' 64 weights; workspaces are rounded up to 256 bytes, one share of them
            assert ssd.block.gated_norm_backward_workspace_bytes(rows, F - F % 64, 64) // 256 * _held(F - F % 64) * CHAIN >= rows, rows


@pytest.mark.gpu
def test_many_rows_whose_roundings_agree():
    """2^26 rows that each add p = 1 + 2^-15 - 2^-22: between 512 and 1024 p a float32 sum loses nearly half a unit with each
    of them. In a chain of n = 256 terms the sums round n times, by U each at most; the 16 rows of a workgroup and the result
    round 17 times more, and the gates here are exact but for some 4 roundings of a term."""
    dev, rows, F = "cuda:0", 1 << 26, 8
    p = 1 + 2.0 ** -15 - 2.0 ** -22
    bar = (CHAIN + 16 + 1 + 4) * U * rows * p
    ones, grad = torch.ones(rows, F, device=dev), torch.full((rows, F), p, device=dev)
    w, r = torch.ones(F, device=dev), torch.ones(rows, device=dev)
    # every row's values are the same: what the second norm hands back is 0, and the residual's gradient alone is left
    g = ssd.block_norm_backward(ones, ones, w, w, r, r, grad, grad_residual=grad)
    for got in (g.post_weight, g.pre_weight):
        assert (got.double() - rows * p).abs().max().item() <= bar
    del g
    # silu(32) is 32 to 14 digits
    g = ssd.gated_norm_backward(ones / 32, ones * 32, w, r[:, None], grad)
    assert (g.weight.double() - rows * p).abs().max().item() <= bar
