"""Host emulation of the gated delta rule (TEST INFRASTRUCTURE): as ops_emu_harness, for ssd_delta_api.hip."""

import ctypes
import os
import subprocess

import numpy as np

import ops_emu_harness as base
from ops_emu_harness import KIND, SIZE, Guarded, get, p, put, space, strided


def build(out_dir):
    out = os.path.join(out_dir, "libdelta_emu.so")
    subprocess.run([base.CLANG, "-x", "c++", "-std=c++17", "-I" + base.EMU, "-I" + base.CSRC,
                    "-I" + os.path.join(base.ROOT, "include"), "-O1", "-g", "-fPIC", "-shared", "-Wno-psabi",
                    os.path.join(base.EMU, "delta_emu_lib.cpp"), "-o", out], check=True)
    return out


def load(path):
    from complex_chunkwise_ssd_amd import block
    lib = ctypes.CDLL(path)
    block.declare_delta(lib)
    lib.emu_set_shuffle_seed.argtypes = [ctypes.c_ulonglong]
    lib.emu_set_shuffle_seed.restype = None
    return lib


def _inputs(q, k, v, g, beta, kind, pad, lengths):
    """The buffers and the arguments up to the sizes; rows of heads lie `pad` elements apart."""
    (B, T, Hk, Dk), (Hv, Dv) = q.shape, v.shape[2:]
    bufs, args = [], []
    for w in (q, k, v):
        flat = np.asarray(w).reshape(B, T, -1)
        bufs.append(strided(flat, kind, flat.shape[-1] + pad))
        args += [p(bufs[-1]), flat.shape[-1] + pad]
    for w in (g, beta):
        bufs.append(put(w, "f32"))
        args.append(p(bufs[-1]))
    N = None if lengths is None else Guarded(4 * B, 4).write(np.asarray(lengths, np.int32).tobytes())
    return bufs + [N], args, (B, T, Hk, Hv, Dk, Dv), N


def delta(lib, q, k, v, g, beta, scale, kind, init=None, lengths=None, states=False, pad=0, in_place=False):
    held, args, sizes, N = _inputs(q, k, v, g, beta, kind, pad, lengths)
    B, T, Hk, Hv, Dk, Dv = sizes
    state, chunks = (B, Hv, Dk, Dv), (B, -(-T // 64), Hv, Dk, Dv)
    I = put(init, "f32")
    o = Guarded(v.size * SIZE[kind], SIZE[kind])
    fin = I if in_place else Guarded(int(np.prod(state)) * 4, 4)
    cs = Guarded(int(np.prod(chunks)) * 4, 4) if states else None
    n = lib.ssd_gated_delta_workspace_bytes(*sizes, KIND[kind])
    ws = space(n)
    rc = lib.ssd_gated_delta(*args, scale, KIND[kind], *sizes, p(I), p(N), p(o), p(fin), p(cs), p(ws), n, None)
    assert rc == 0, rc
    return get(o, kind, v.shape), get(fin, "f32", state), get(cs, "f32", chunks) if states else None


def delta_backward(lib, q, k, v, g, beta, scale, kind, states, go, gfinal=None, lengths=None, pad=0):
    held, args, sizes, N = _inputs(q, k, v, g, beta, kind, pad, lengths)
    B, T, Hk, Hv, Dk, Dv = sizes
    S, G, F = put(states, "f32"), put(go, kind), put(gfinal, "f32")
    shapes = [(q.shape, kind), (q.shape, kind), (v.shape, kind), (g.shape, "f32"), (g.shape, "f32"),
              ((B, Hv, Dk, Dv), "f32")]
    out = [Guarded(int(np.prod(s)) * SIZE[t], SIZE[t]) for s, t in shapes]
    n = lib.ssd_gated_delta_backward_workspace_bytes(*sizes, KIND[kind])
    ws = space(n)
    rc = lib.ssd_gated_delta_backward(*args, scale, KIND[kind], *sizes, p(S), p(N), p(G), p(F), *map(p, out), p(ws), n,
                                      None)
    assert rc == 0, rc
    return [get(b, t, s) for b, (s, t) in zip(out, shapes)]
