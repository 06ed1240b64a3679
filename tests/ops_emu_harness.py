"""Host emulation of the operators around the scan (TEST INFRASTRUCTURE): the unchanged C-ABI
and kernel sources built against the emulated device headers. Every buffer that a call
gets ends at a page that cannot be touched, so that an access past its end stops the process."""

import ctypes
import mmap
import os
import subprocess
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
EMU = os.path.join(HERE, "emu")
CSRC = os.path.join(ROOT, "complex_chunkwise_ssd_amd", "csrc")
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
CLANG = "/opt/rocm/llvm/bin/clang++"

_libc = ctypes.CDLL(None, use_errno=True)
_libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
F32, BF16 = 0, 1
KIND = {"f32": F32, "bf16": BF16}


def build(out_dir):
    out = os.path.join(out_dir, "libops_emu.so")
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-I" + EMU, "-I" + CSRC,
                    "-I" + os.path.join(ROOT, "include"), "-O1", "-g", "-fPIC", "-shared", "-Wno-psabi",
                    os.path.join(EMU, "ops_emu_lib.cpp"), "-o", out], check=True)
    return out


def load(path):
    from complex_chunkwise_ssd_amd import ops
    lib = ctypes.CDLL(path)
    ops.declare(lib)
    lib.emu_set_shuffle_seed.argtypes = [ctypes.c_ulonglong]
    lib.emu_set_shuffle_seed.restype = None
    return lib


class Guarded:
    """`n` bytes that end (up to `align` - 1 bytes of slack) at a page without access."""

    def __init__(self, n, align=1, fill=0xff):
        page = mmap.PAGESIZE
        body = max(page, -(-n // page) * page)
        self.map = mmap.mmap(-1, body + page)
        base = ctypes.addressof(ctypes.c_char.from_buffer(self.map))
        if _libc.mprotect(base + body, page, 0):
            raise OSError("mprotect")
        self.at = base + (body - n) // align * align
        self.n = n
        ctypes.memset(self.at, fill, n)

    def write(self, data):
        ctypes.memmove(self.at, data, len(data))
        return self

    def read(self, dtype, shape):
        return np.frombuffer(ctypes.string_at(self.at, self.n), dtype)[:int(np.prod(shape))].reshape(shape).copy()


def _bytes(v, kind):
    """Values as the library takes them."""
    if kind == "bf16":
        return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16).tobytes()
    if kind == "u8":
        return np.asarray(v, np.uint8).tobytes()
    return np.asarray(v, np.float32).tobytes()


SIZE = {"f32": 4, "bf16": 2, "u8": 1}


def put(v, kind, align=None):
    if v is None:
        return None
    data = _bytes(v, kind)
    return Guarded(len(data), align or SIZE[kind]).write(data)


def strided(v, kind, stride, offset=0):
    """v (..., F) with rows `stride` elements apart, NaN patterns between them."""
    v = np.asarray(v)
    rows, F = int(np.prod(v.shape[:-1])), v.shape[-1]
    e = SIZE[kind]
    g = Guarded(((rows - 1) * stride + F + offset) * e if rows else 0, e)
    src = _bytes(v, kind)
    for r in range(rows):
        ctypes.memmove(g.at + (offset + r * stride) * e, src[r * F * e:(r + 1) * F * e], F * e)
    g.at += offset * e
    g.n -= offset * e
    return g


def get(g, kind, shape):
    if kind == "bf16":
        return (g.read(np.uint16, shape).astype(np.uint32) << 16).view(np.float32)
    return g.read(np.uint8 if kind == "u8" else np.float32, shape)


def p(g):
    return None if g is None else g.at


def space(n):
    return Guarded(n, 256) if n else None


def gated(lib, x, gi, gr, lam, k, kind, init=None, lengths=None, states=False, pad=0, in_place=False):
    B, T, C = x.shape
    st = C + pad
    xs, gis, grs = (strided(v, kind, st) for v in (x, gi, gr))
    L, I = put(lam, "f32"), put(init, "f32")
    N = None if lengths is None else Guarded(4 * B, 4).write(np.asarray(lengths, np.int32).tobytes())
    h = Guarded(B * T * C * SIZE[kind], SIZE[kind])
    fin = I if in_place else Guarded(B * C * 4, 4)
    cs = Guarded(B * -(-T // 64) * C * 4, 4) if states else None
    n = lib.ssd_gated_scan_workspace_bytes(B, T, C, KIND[kind])
    ws = space(n)
    rc = lib.ssd_gated_scan(p(xs), st, p(gis), st, p(grs), st, p(L), k, KIND[kind], B, T, C, p(I), p(N),
                            p(h), p(fin), p(cs), p(ws), n, None)
    assert rc == 0, rc
    return (get(h, kind, (B, T, C)), get(fin, "f32", (B, C)),
            get(cs, "f32", (B, -(-T // 64), C)) if states else None)


def gated_backward(lib, x, gi, gr, lam, k, kind, cs, gh, gfinal=None, lengths=None, pad=0):
    B, T, C = x.shape
    st = C + pad
    xs, gis, grs = (strided(v, kind, st) for v in (x, gi, gr))
    L, S, G, GF = put(lam, "f32"), put(cs, "f32"), put(gh, kind), put(gfinal, "f32")
    N = None if lengths is None else Guarded(4 * B, 4).write(np.asarray(lengths, np.int32).tobytes())
    o = [Guarded(B * T * C * SIZE[kind], SIZE[kind]) for _ in range(3)]
    gl, gi0 = Guarded(C * 4, 4), Guarded(B * C * 4, 4)
    n = lib.ssd_gated_scan_backward_workspace_bytes(B, T, C, KIND[kind])
    ws = space(n)
    rc = lib.ssd_gated_scan_backward(p(xs), st, p(gis), st, p(grs), st, p(L), k, KIND[kind], B, T, C, p(S),
                                     p(N), p(G), p(GF), p(o[0]), p(o[1]), p(o[2]), p(gl), p(gi0), p(ws),
                                     n, None)
    assert rc == 0, rc
    return [get(v, kind, (B, T, C)) for v in o] + [get(gl, "f32", (C,)), get(gi0, "f32", (B, C))]


def norm(lib, x, res, w, eps, kind, y=True, fp8=True, pad=0, in_place=False):
    R, F = x.shape
    X = strided(x, kind, F + pad)
    Z = None if res is None else strided(res, kind, F if in_place else F + pad)
    W = put(w, "f32")
    e = SIZE[kind]
    Y = Guarded(R * F * e, e) if y else None
    S = None if res is None else Z if in_place else Guarded(R * F * e, e)
    Q, C = (Guarded(R * F, 1), Guarded(-(-F // 128) * R * 4, 4)) if fp8 else (None, None)
    D = Guarded(R * 4, 4)
    rc = lib.ssd_rms_norm(p(X), F + pad, p(Z), F if in_place else F + pad, p(W), KIND[kind], R, F, eps,
                          p(Y), p(S), p(Q), p(C), p(D), None)
    assert rc == 0, rc
    return dict(y=get(Y, kind, (R, F)) if y else None, s=None if res is None else get(S, kind, (R, F)),
                q=get(Q, "u8", (R, F)) if fp8 else None,
                scale=get(C, "f32", (-(-F // 128), R)) if fp8 else None, rstd=get(D, "f32", (R,)))


def norm_backward(lib, s, w, rstd, gy, gs, kind, pad=0):
    R, F = s.shape
    S, G = strided(s, kind, F + pad), strided(gy, kind, F + pad)
    Z = None if gs is None else strided(gs, kind, F + pad)
    W, D = put(w, "f32"), put(rstd, "f32")
    e = SIZE[kind]
    X, GW = Guarded(R * F * e, e), Guarded(F * 4, 4)
    n = lib.ssd_rms_norm_backward_workspace_bytes(R, F)
    ws = space(n)
    rc = lib.ssd_rms_norm_backward(p(S), F + pad, p(W), p(D), p(G), F + pad, p(Z), F + pad, KIND[kind], R, F,
                                   p(X), p(GW), p(ws), n, None)
    assert rc == 0, rc
    return get(X, kind, (R, F)), get(GW, "f32", (F,))


def quantise(lib, x, kind, block_rows, turn, pad=0, q_pad=0):
    R, C = x.shape
    X = strided(x, kind, C + pad)
    qr, qc = (C, R) if turn else (R, C)
    st = qc + q_pad
    Q = Guarded((qr - 1) * st + qc, 1)
    shape = (-(-qc // 128), qr) if block_rows == 1 else (-(-qr // 128), -(-qc // 128))
    S = Guarded(4 * shape[0] * shape[1], 4)
    rc = lib.ssd_fp8_quantise(p(X), C + pad, KIND[kind], R, C, block_rows, int(turn), p(Q), st, p(S), None)
    assert rc == 0, rc
    raw = Q.read(np.uint8, (Q.n,))
    rows = np.stack([raw[r * st:r * st + qc] for r in range(qr)])
    for r in range(qr - 1):  # between the rows nothing is written
        assert (raw[r * st + qc:(r + 1) * st] == 0xff).all()
    return rows, get(S, "f32", shape)


def matmul(lib, a, sa, b, sb, block_rows, out, a_pad=0, b_pad=0, out_pad=0, align=16):
    """a (M, K), b (N, K) e4m3 bytes."""
    M, K = a.shape
    N = b.shape[0]

    def rows(v, pad):  # the end of the last row, rounded up to `align`, is the end of the buffer
        st = v.shape[1] + pad
        g = Guarded((v.shape[0] - 1) * st + v.shape[1], align)
        for r in range(v.shape[0]):
            ctypes.memmove(g.at + r * st, np.ascontiguousarray(v[r], np.uint8).tobytes(), v.shape[1])
        return g
    A, B = rows(a, a_pad), rows(b, b_pad)
    SA, SB = put(sa, "f32"), put(sb, "f32")
    e = SIZE[out]
    O = Guarded(((M - 1) * (N + out_pad) + N) * e, e)
    on16 = int((A.at | B.at | (K + a_pad) | (K + b_pad)) % 16 == 0)
    n = lib.ssd_fp8_matmul_workspace_bytes(M, N, K, block_rows, KIND[out], on16)
    ws = space(n)
    rc = lib.ssd_fp8_matmul(p(A), K + a_pad, p(SA), p(B), K + b_pad, p(SB), M, N, K, block_rows, KIND[out],
                            p(O), N + out_pad, p(ws), n, None)
    assert rc == 0, rc
    flat = get(O, out, (O.n // e,))
    return np.stack([flat[m * (N + out_pad):m * (N + out_pad) + N] for m in range(M)])
