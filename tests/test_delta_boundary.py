"""The gated delta rule's C ABI and Python layer on the CPU: what is refused, before anything is launched.
Only refused calls and calls without work: their addresses are made up."""

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


SIZES = dict(scale=0.1, dt=1, B=2, T=100, Hk=2, Hv=4, Dk=16, Dv=32)
ROWS = dict(q=_at(0), qs=32, k=_at(1), ks=32, v=_at(2), vs=128, g=_at(3), b=_at(4))


def _fwd(lib, **kw):
    a = dict(**ROWS, **SIZES, i=_at(5), n=_at(6), o=_at(7), f=_at(8), cs=_at(9), ws=_at(10), wn=1 << 30)
    a.update(kw)
    return lib.ssd_gated_delta(*a.values(), None)


def _bwd(lib, **kw):
    a = dict(**ROWS, **SIZES, cs=_at(5), n=_at(6), go=_at(7), gf=_at(8), gq=_at(9), gk=_at(10), gv=_at(11), gg=_at(12),
             gb=_at(13), g0=_at(14), ws=_at(15), wn=1 << 30)
    a.update(kw)
    return lib.ssd_gated_delta_backward(*a.values(), None)


SHAPES = (dict(B=-1), dict(T=-1), dict(Hk=0), dict(Hv=0), dict(Dk=0), dict(Dv=0), dict(Hk=3), dict(Hv=5), dict(Hv=1), dict(dt=2),
          dict(dt=-1), dict(qs=31), dict(ks=31), dict(vs=127), dict(scale=float("nan")), dict(scale=float("inf")),
          dict(scale=-2e30))


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_shapes(lib, call):
    for bad in SHAPES:
        assert call(lib, **bad) == ssd.SSD_ERR_SHAPE, bad
    assert call(lib, Dk=129, qs=1 << 20, ks=1 << 20) == ssd.SSD_ERR_BLOCK_DIMS
    assert call(lib, Dv=257, vs=1 << 20) == ssd.SSD_ERR_BLOCK_DIMS
    for bad in (dict(T=(1 << 30) + 1), dict(B=(1 << 24) + 1), dict(Hv=1 << 17, Hk=1, vs=1 << 30), dict(qs=1 << 60),
                dict(B=1 << 22), dict(B=1 << 20, T=300), dict(B=1 << 20, Dv=256, vs=1024)):
        assert call(lib, **bad) == ssd.SSD_ERR_UNSUPPORTED, bad


def test_forward_refusals(lib):
    for name in ("q", "k", "v", "g", "b", "o"):
        assert _fwd(lib, **{name: None}) == ssd.SSD_ERR_NULL, name
    for name, off in (("q", 1), ("k", 1), ("v", 1), ("g", 2), ("b", 2), ("i", 2), ("n", 2), ("o", 1), ("f", 2), ("cs", 2)):
        assert _fwd(lib, **{name: _at(20, off)}) == ssd.SSD_ERR_ALIGN, name
    for name in ("q", "k", "v"):
        assert _fwd(lib, dt=0, **{name: _at(20, 2)}) == ssd.SSD_ERR_ALIGN, name
    for a in ("o", "f", "cs", "ws"):
        for b in range(7):
            if (a, b) != ("f", 5):
                assert _fwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    for a, b in (("f", 7), ("cs", 8), ("ws", 9), ("o", 8)):
        assert _fwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    assert _fwd(lib, f=_at(5, 4)) == ssd.SSD_ERR_ALIAS          # in place, but not quite
    assert _fwd(lib, f=_at(5), o=_at(5, 256)) == ssd.SSD_ERR_ALIAS
    assert _fwd(lib, ws=None) == ssd.SSD_ERR_WORKSPACE
    assert _fwd(lib, ws=_at(10, 8)) == ssd.SSD_ERR_ALIGN
    need = lib.ssd_gated_delta_workspace_bytes(2, 100, 2, 4, 16, 32, 1)
    assert need > 0 and _fwd(lib, wn=need - 1) == ssd.SSD_ERR_WORKSPACE
    assert lib.ssd_gated_delta_workspace_bytes(2, 8, 2, 4, 16, 32, 1) == 0      # a few tokens need none
    for bad in ((-1, 100, 2, 4, 16, 32, 1), (2, 100, 3, 4, 16, 32, 1), (2, 100, 2, 4, 129, 32, 1), (2, 100, 2, 4, 16, 32, 7)):
        assert lib.ssd_gated_delta_workspace_bytes(*bad) == 0, bad
    assert _fwd(lib, B=0, q=None, o=None) == ssd.SSD_OK
    assert _fwd(lib, T=0, q=None, o=None, f=None) == ssd.SSD_OK
    assert _fwd(lib, T=0, f=_at(5)) == ssd.SSD_OK               # the state stays where it is
    assert _fwd(lib, T=0, f=_at(5, 4)) == ssd.SSD_ERR_ALIAS


def test_backward_refusals(lib):
    for name in ("q", "k", "v", "g", "b", "cs", "go", "gq", "gk", "gv", "gg", "gb"):
        assert _bwd(lib, **{name: None}) == ssd.SSD_ERR_NULL, name
    for name, off in (("q", 1), ("go", 1), ("gq", 1), ("gk", 1), ("gv", 1), ("cs", 2), ("gf", 2), ("gg", 2), ("gb", 2),
                      ("g0", 2), ("n", 2)):
        assert _bwd(lib, **{name: _at(20, off)}) == ssd.SSD_ERR_ALIGN, name
    outs = ("gq", "gk", "gv", "gg", "gb", "g0", "ws")
    for a in outs:
        for b in range(9):
            assert _bwd(lib, **{a: _at(b)}) == ssd.SSD_ERR_ALIAS, (a, b)
    for i, a in enumerate(outs[1:]):
        assert _bwd(lib, **{a: _at(9 + i)}) == ssd.SSD_ERR_ALIAS, a
    assert _bwd(lib, ws=None) == ssd.SSD_ERR_WORKSPACE
    assert _bwd(lib, ws=_at(15, 8)) == ssd.SSD_ERR_ALIGN
    need = lib.ssd_gated_delta_backward_workspace_bytes(2, 100, 2, 4, 16, 32, 1)
    assert need > 0 and _bwd(lib, wn=need - 1) == ssd.SSD_ERR_WORKSPACE
    assert _bwd(lib, B=0, q=None, gq=None) == ssd.SSD_OK
    assert _bwd(lib, T=0, q=None, gq=None, g0=None) == ssd.SSD_OK
    assert _bwd(lib, T=0, g0=_at(8, 4)) == ssd.SSD_ERR_ALIAS


def test_python_layer_rejects_bad_tensors():
    x = torch.zeros(2, 4, 2, 8)
    g = torch.zeros(2, 4, 2)
    with pytest.raises(ValueError):
        ssd.gated_delta(x, x, x, g, g)          # CPU tensors
    with pytest.raises(ValueError):
        ssd.gated_delta_backward(x, x, x, g, g, x, x)


def test_token_strides():
    stride = ssd.block._binding().token_stride
    rows = torch.zeros(3, 5, 40)
    heads = lambda t: t.unflatten(-1, (2, 8))  # noqa: E731
    assert stride(torch.zeros(3, 5, 2, 8)) == 16 and stride(heads(rows[..., 8:24])) == 40
    assert stride(heads(rows[:1, :, 8:24])) == 40 and stride(heads(rows[:, :1, 8:24].contiguous())) == 16
    assert stride(heads(rows[:, :1, 8:24])) == 200      # one token a row: the rows lie 200 apart
    assert stride(heads(rows[:1, :1, 8:24])) == 16
    for bad in (torch.zeros(3, 2, 5, 8).transpose(1, 2), heads(rows[:, :4, 8:24]), heads(rows[..., ::2][..., :16]),
                torch.zeros(3, 1, 2, 8).expand(3, 5, 2, 8), torch.zeros(3, 5, 1, 8).expand(3, 5, 2, 8)):
        with pytest.raises(ValueError):
            stride(bad)


def test_chunk_matches_the_header():
    text = open(ssd.HEADER).read()
    assert "#define SSD_DELTA_CHUNK %d" % ssd.DELTA_CHUNK in text


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_launches_of_2_to_the_32_threads(lib, call):
    # 129 to 192 columns are walked in two blocks of 512 threads: 2^22 heads are 2^32 threads, one less is not refused
    # for its size (and stopped by the missing q)
    wide = dict(T=9, Hk=1, Hv=1, Dk=65, Dv=129, qs=65, ks=65, vs=129, q=None)
    assert call(lib, B=1 << 22, **wide) == ssd.SSD_ERR_UNSUPPORTED
    assert call(lib, B=(1 << 22) - 1, **wide) == ssd.SSD_ERR_NULL
