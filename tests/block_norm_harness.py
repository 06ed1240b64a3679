"""Host emulation of the norms around a block (TEST INFRASTRUCTURE): as ops_emu_harness, for ssd_block_api.hip."""

import ctypes
import os
import subprocess

import ops_emu_harness as base
from ops_emu_harness import KIND, SIZE, Guarded, get, p, put, space, strided


def build(out_dir):
    out = os.path.join(out_dir, "libblock_emu.so")
    subprocess.run([base.CLANG, "-x", "c++", "-std=c++17", "-I" + base.EMU, "-I" + base.CSRC,
                    "-I" + os.path.join(base.ROOT, "include"), "-O1", "-g", "-fPIC", "-shared", "-Wno-psabi",
                    os.path.join(base.EMU, "block_emu_lib.cpp"), "-o", out], check=True)
    return out


def load(path):
    from complex_chunkwise_ssd_amd import block
    lib = ctypes.CDLL(path)
    block.declare_norms(lib)
    lib.emu_set_shuffle_seed.argtypes = [ctypes.c_ulonglong]
    lib.emu_set_shuffle_seed.restype = None
    return lib


def _eight(R, F, fp8):
    return (Guarded(R * F, 1), Guarded(-(-F // 128) * R * 4, 4)) if fp8 else (None, None)


def gated_norm(lib, x, z, w, eps, kind, y=True, fp8=True, pad=0):
    (R, F), D, e = x.shape, len(w), SIZE[kind]
    X, Z, W = strided(x, kind, F + pad), strided(z, kind, F + pad), put(w, "f32")
    Y = Guarded(R * F * e, e) if y else None
    Q, C = _eight(R, F, fp8)
    S = Guarded(R * (F // D) * 4, 4)
    rc = lib.ssd_gated_norm(p(X), F + pad, p(Z), F + pad, p(W), KIND[kind], R, F, D, eps, p(Y), p(Q), p(C), p(S), None)
    assert rc == 0, rc
    return dict(y=get(Y, kind, (R, F)) if y else None, q=get(Q, "u8", (R, F)) if fp8 else None,
                scale=get(C, "f32", (-(-F // 128), R)) if fp8 else None, rstd=get(S, "f32", (R, F // D)))


def gated_norm_backward(lib, x, z, w, rstd, gy, kind, pad=0):
    (R, F), D, e = x.shape, len(w), SIZE[kind]
    X, Z, G = (strided(v, kind, F + pad) for v in (x, z, gy))
    W, S = put(w, "f32"), put(rstd, "f32")
    gx, gz, gw = Guarded(R * F * e, e), Guarded(R * F * e, e), Guarded(D * 4, 4)
    n = lib.ssd_gated_norm_backward_workspace_bytes(R, F, D)
    ws = space(n)
    rc = lib.ssd_gated_norm_backward(p(X), F + pad, p(Z), F + pad, p(W), p(S), p(G), F + pad, KIND[kind], R, F, D,
                                     p(gx), p(gz), p(gw), p(ws), n, None)
    assert rc == 0, rc
    return get(gx, kind, (R, F)), get(gz, kind, (R, F)), get(gw, "f32", (D,))


def block_norm(lib, x, res, w1, w2, alpha, eps, kind, y=True, fp8=True, pad=0, in_place=False):
    (R, F), e = x.shape, SIZE[kind]
    rs = F if in_place else F + pad
    X, Z, W1, W2 = strided(x, kind, F + pad), strided(res, kind, rs), put(w1, "f32"), put(w2, "f32")
    Y = Guarded(R * F * e, e) if y else None
    S = Z if in_place else Guarded(R * F * e, e)
    Q, C = _eight(R, F, fp8)
    A, B = Guarded(R * 4, 4), Guarded(R * 4, 4)
    rc = lib.ssd_block_norm(p(X), F + pad, p(Z), rs, p(W1), p(W2), alpha, KIND[kind], R, F, eps, p(Y), p(S), p(Q), p(C),
                            p(A), p(B), None)
    assert rc == 0, rc
    return dict(y=get(Y, kind, (R, F)) if y else None, s=get(S, kind, (R, F)), q=get(Q, "u8", (R, F)) if fp8 else None,
                scale=get(C, "f32", (-(-F // 128), R)) if fp8 else None, post=get(A, "f32", (R,)),
                pre=get(B, "f32", (R,)))


def block_norm_backward(lib, x, s, w1, w2, r1, r2, alpha, gy, gs, kind, pad=0):
    (R, F), e = x.shape, SIZE[kind]
    X, S, G = (strided(v, kind, F + pad) for v in (x, s, gy))
    Z = None if gs is None else strided(gs, kind, F + pad)
    W1, W2, A, B = (put(v, "f32") for v in (w1, w2, r1, r2))
    out = [Guarded(R * F * e, e), Guarded(R * F * e, e), Guarded(F * 4, 4), Guarded(F * 4, 4)]
    n = lib.ssd_block_norm_backward_workspace_bytes(R, F)
    ws = space(n)
    rc = lib.ssd_block_norm_backward(p(X), F + pad, p(S), F + pad, p(W1), p(W2), p(A), p(B), alpha, p(G), F + pad, p(Z),
                                     F + pad, KIND[kind], R, F, *map(p, out), p(ws), n, None)
    assert rc == 0, rc
    return [get(o, k, (R, F) if i < 2 else (F,)) for i, (o, k) in enumerate(zip(out, (kind, kind, "f32", "f32")))]
