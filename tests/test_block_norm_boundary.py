"""The C ABI of the norms around a block, and their Python layer, on the CPU: what is refused, before anything is
launched. Only refused calls and calls without work: their addresses are made up."""

import ctypes
import os

import pytest
import torch

import complex_chunkwise_ssd_amd as ssd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIBPATH):
        from complex_chunkwise_ssd_amd import build
        build.build()
    return ssd.load_library()


def _at(k, off=0):
    """Made-up device addresses, 1 TiB apart."""
    return ctypes.c_void_p((k + 1 << 40) + off)


def _gated(lib, **kw):
    a = dict(x=_at(0), xs=32, z=_at(1), zs=32, w=_at(2), dt=1, rows=4, F=32, D=8, eps=1e-6, y=_at(3), q=_at(4), sc=_at(5),
             rstd=_at(6))
    a.update(kw)
    return lib.ssd_gated_norm(*a.values(), None)


def test_gated_norm_refusals(lib):
    for bad in (dict(rows=-1), dict(F=0), dict(D=0), dict(D=12), dict(xs=31), dict(zs=31), dict(dt=2), dict(eps=-1.0),
                dict(eps=float("nan"))):
        assert _gated(lib, **bad) == ssd.SSD_ERR_SHAPE, bad
    for bad in (dict(D=4), dict(F=16392, xs=1 << 15, zs=1 << 15), dict(rows=1 << 31), dict(xs=1 << 60)):
        assert _gated(lib, **bad) == ssd.SSD_ERR_UNSUPPORTED, bad
    for bad in (dict(x=None), dict(z=None), dict(w=None), dict(y=None, q=None), dict(sc=None)):
        assert _gated(lib, **bad) == ssd.SSD_ERR_NULL, bad
    for name, off in (("x", 1), ("z", 1), ("w", 2), ("y", 1), ("sc", 2), ("rstd", 2)):
        assert _gated(lib, **{name: _at(20, off)}) == ssd.SSD_ERR_ALIGN, name
    for a, b in (("y", 0), ("y", 1), ("y", 2), ("q", 0), ("q", 3), ("sc", 1), ("sc", 4), ("rstd", 5), ("rstd", 2)):
        assert _gated(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    assert _gated(lib, rows=0, x=None, y=None, q=None) == ssd.SSD_OK


def _gated_bwd(lib, **kw):
    a = dict(x=_at(0), xs=32, z=_at(1), zs=32, w=_at(2), rstd=_at(3), gy=_at(4), gys=32, dt=1, rows=4, F=32, D=8, gx=_at(5),
             gz=_at(6), gw=_at(7), ws=_at(8), wn=1 << 20)
    a.update(kw)
    return lib.ssd_gated_norm_backward(*a.values(), None)


def test_gated_norm_backward_refusals(lib):
    for bad in (dict(rows=-1), dict(F=0), dict(D=12), dict(xs=31), dict(zs=31), dict(gys=31), dict(dt=-1)):
        assert _gated_bwd(lib, **bad) == ssd.SSD_ERR_SHAPE, bad
    for bad in (dict(D=4), dict(gys=1 << 60)):
        assert _gated_bwd(lib, **bad) == ssd.SSD_ERR_UNSUPPORTED, bad
    for name in ("x", "z", "w", "rstd", "gy", "gx", "gz", "gw"):
        assert _gated_bwd(lib, **{name: None}) == ssd.SSD_ERR_NULL, name
    for name, off in (("x", 1), ("gy", 1), ("gx", 1), ("gz", 1), ("gw", 2), ("rstd", 2)):
        assert _gated_bwd(lib, **{name: _at(20, off)}) == ssd.SSD_ERR_ALIGN, name
    for a in ("gx", "gz", "gw", "ws"):
        for b in range(5):
            assert _gated_bwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    for a, b in (("gz", 5), ("gw", 6), ("ws", 7)):
        assert _gated_bwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    assert _gated_bwd(lib, ws=None) == ssd.SSD_ERR_WORKSPACE and _gated_bwd(lib, wn=16) == ssd.SSD_ERR_WORKSPACE
    assert _gated_bwd(lib, ws=_at(8, 8)) == ssd.SSD_ERR_ALIGN
    assert lib.ssd_gated_norm_backward_workspace_bytes(4, 32, 12) == 0


def _block(lib, **kw):
    a = dict(x=_at(0), xs=32, r=_at(1), rs=32, w1=_at(2), w2=_at(3), al=0.5, dt=1, rows=4, F=32, eps=1e-6, y=_at(4), s=_at(5),
             q=_at(6), sc=_at(7), r1=_at(8), r2=_at(9))
    a.update(kw)
    return lib.ssd_block_norm(*a.values(), None)


def test_block_norm_refusals(lib):
    for bad in (dict(rows=-1), dict(F=0), dict(xs=31), dict(rs=31), dict(dt=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(al=float("nan")), dict(al=float("inf")), dict(al=-2e30)):
        assert _block(lib, **bad) == ssd.SSD_ERR_SHAPE, bad
    for bad in (dict(F=16385, xs=1 << 15, rs=1 << 15), dict(rs=1 << 60)):
        assert _block(lib, **bad) == ssd.SSD_ERR_UNSUPPORTED, bad
    for bad in (dict(x=None), dict(r=None), dict(w1=None), dict(w2=None), dict(s=None), dict(y=None, q=None), dict(sc=None)):
        assert _block(lib, **bad) == ssd.SSD_ERR_NULL, bad
    for name, off in (("x", 1), ("r", 1), ("w1", 2), ("w2", 2), ("y", 1), ("s", 1), ("sc", 2), ("r1", 2), ("r2", 2)):
        assert _block(lib, **{name: _at(20, off)}) == ssd.SSD_ERR_ALIGN, name
    for a in ("y", "s", "q", "sc", "r1", "r2"):
        for b in range(4):
            if (a, b) != ("s", 1):
                assert _block(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    for a, b in (("s", 4), ("q", 5), ("sc", 6), ("r1", 7), ("r2", 8)):
        assert _block(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    assert _block(lib, s=_at(1), rs=33) == ssd.SSD_ERR_ALIAS      # in place only where the rows are dense
    assert _block(lib, rows=0, x=None, s=None) == ssd.SSD_OK


def _block_bwd(lib, **kw):
    a = dict(x=_at(0), xs=32, s=_at(1), ss=32, w1=_at(2), w2=_at(3), r1=_at(4), r2=_at(5), al=0.5, gy=_at(6), gys=32, gs=_at(7),
             gss=32, dt=1, rows=4, F=32, gx=_at(8), gr=_at(9), g1=_at(10), g2=_at(11), ws=_at(12), wn=1 << 20)
    a.update(kw)
    return lib.ssd_block_norm_backward(*a.values(), None)


def test_block_norm_backward_refusals(lib):
    for bad in (dict(rows=-1), dict(F=0), dict(xs=31), dict(ss=31), dict(gys=31), dict(gss=31), dict(dt=2), dict(al=float("nan"))):
        assert _block_bwd(lib, **bad) == ssd.SSD_ERR_SHAPE, bad
    for name in ("x", "s", "w1", "w2", "r1", "r2", "gy", "gx", "gr", "g1", "g2"):
        assert _block_bwd(lib, **{name: None}) == ssd.SSD_ERR_NULL, name
    for name, off in (("x", 1), ("gy", 1), ("gs", 1), ("gx", 1), ("gr", 1), ("g1", 2), ("g2", 2), ("r1", 2)):
        assert _block_bwd(lib, **{name: _at(20, off)}) == ssd.SSD_ERR_ALIGN, name
    for a in ("gx", "gr", "g1", "g2", "ws"):
        for b in range(8):
            assert _block_bwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    for a, b in (("gr", 8), ("g1", 9), ("g2", 10), ("ws", 11)):
        assert _block_bwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    assert _block_bwd(lib, ws=None) == ssd.SSD_ERR_WORKSPACE and _block_bwd(lib, wn=16) == ssd.SSD_ERR_WORKSPACE
    assert _block_bwd(lib, ws=_at(12, 8)) == ssd.SSD_ERR_ALIGN
    assert _block_bwd(lib, rows=0, g2=_at(10)) == ssd.SSD_ERR_ALIAS


def test_python_layer_rejects_bad_tensors():
    x, w = torch.zeros(2, 4, 8), torch.zeros(8)
    for call in (lambda: ssd.gated_norm(x, x, w), lambda: ssd.gated_norm_backward(x, x, w, w, x),
                 lambda: ssd.block_norm(x, x, w, w), lambda: ssd.block_norm_backward(x, x, w, w, w, w, x)):
        with pytest.raises(ValueError):          # CPU tensors
            call()


def test_the_binding_calls_the_library_of_the_package():
    at = lambda name: ctypes.cast(getattr(ssd.load_library(), name), ctypes.c_void_p).value  # noqa: E731
    bound = ssd.block._binding().bound()
    assert len(bound) == 10 and all(address == at(name) for name, address in bound.items())
