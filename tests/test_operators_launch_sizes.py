"""The operators' C ABI on the CPU: a call whose launch would have 2^32 threads or more, which HIP
does not take, is refused before anything is launched. Only refused calls: their addresses are
made up."""

import ctypes
import os

import pytest

import complex_chunkwise_ssd_amd as ssd

UNSUPPORTED = ssd.SSD_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIBPATH):
        from complex_chunkwise_ssd_amd import build
        build.build()
    return ssd.load_library()


def _at(k):
    """Made-up device addresses, 16 TiB apart."""
    return ctypes.c_void_p(k + 1 << 44)


WS = (_at(30), 1 << 43)


def _gated(lib, B, T, C):
    return lib.ssd_gated_scan(_at(0), C, _at(1), C, _at(2), C, _at(3), 8.0, 0, B, T, C, None, None, _at(4), None, None,
                              *WS, None)


def _gated_backward(lib, B, T, C):
    return lib.ssd_gated_scan_backward(_at(0), C, _at(1), C, _at(2), C, _at(3), 8.0, 0, B, T, C, _at(4), None, _at(5),
                                       None, _at(6), _at(7), _at(8), _at(9), None, *WS, None)


@pytest.mark.parametrize("B,T,C", [(1 << 22, 33, 1), (1 << 24, 64, 2), (1 << 14, 40, 1 << 14), (1 << 12, 100, 1 << 24)])
def test_gated_scan(lib, B, T, C):
    """Workgroups of 1024 threads: 2^22 of them."""
    assert _gated(lib, B, T, C) == UNSUPPORTED
    assert _gated_backward(lib, B, T, C) == UNSUPPORTED


@pytest.mark.parametrize("B,T,C", [(1 << 24, 1, 1 << 8), (1 << 20, 32, 1 << 12), (1 << 8, 1, 1 << 24)])
def test_gated_walk(lib, B, T, C):
    """Workgroups of 64: 2^26."""
    assert _gated(lib, B, T, C) == UNSUPPORTED


@pytest.mark.parametrize("rows,cols,block_rows,turn", [(1 << 30, 1, 1, 0), (1 << 24, 1 << 13, 1, 0), (1 << 31, 1, 128, 0),
                                                       (1, 1 << 31, 1, 1), (1 << 31, 128, 128, 1)])
def test_fp8_quantise(lib, rows, cols, block_rows, turn):
    """Workgroups of 256: 2^24, each 64 blocks of a row or one tile of 128 x 128."""
    assert lib.ssd_fp8_quantise(_at(0), cols, 0, rows, cols, block_rows, turn, _at(1), rows if turn else cols, _at(2),
                                None) == UNSUPPORTED


@pytest.mark.parametrize("M,N,block_rows", [(1 << 30, 1, 128), (1 << 30, 200, 1)])
def test_fp8_matmul(lib, M, N, block_rows):
    """Workgroups of 512 per 128 rows of a: 2^23."""
    assert lib.ssd_fp8_matmul(_at(0), 16, _at(1), _at(2), 16, _at(3), M, N, 16, block_rows, 0, _at(4), N, *WS,
                              None) == UNSUPPORTED
