"""The operators around the scan on the GPU, through the Python entry points: the emulator's
cases against float64 formulas, then what only a GPU shows (captured and replayed calls, other
streams, repeated calls bit for bit, large sizes) and a run of the operators together with
the scan."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import complex_chunkwise_ssd_amd as ssd
import operators_cases as cases
import operators_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}
FP8 = torch.float8_e4m3fn


def _t(v, kind="f32"):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(KIND[kind]).to(DEV)


def _strided(v, kind, pad):
    """v with its rows `pad` elements further apart, NaN between them."""
    t = _t(v, kind)
    if not pad:
        return t
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device=DEV)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _n(t):
    if t is None:
        return None
    torch.cuda.synchronize()
    return t.view(torch.uint8).cpu().numpy() if t.dtype == FP8 else t.float().cpu().numpy()


def _fp8(v, pad=0, align=16):
    t = torch.from_numpy(np.ascontiguousarray(v, np.uint8)).to(DEV)
    R, K = t.shape
    off = 0 if align == 16 else 3
    flat = torch.full((R * (K + pad) + 16,), 0x7f, dtype=torch.uint8, device=DEV)
    view = torch.as_strided(flat, (R, K), (K + pad, 1), off)
    view.copy_(t)
    return view.view(FP8)


class _Gpu:
    """The functions of ops_emu_harness on the GPU."""

    @staticmethod
    def gated(x, gi, gr, lam, k, kind, init=None, lengths=None, states=False, pad=0, in_place=False):
        n = None if lengths is None else torch.from_numpy(lengths).to(DEV)
        i = _t(init)
        r = ssd.gated_scan(_strided(x, kind, pad), _strided(gi, kind, pad), _strided(gr, kind, pad), _t(lam),
                           decay_scale=k, initial_state=i, lengths=n, want_chunk_states=states,
                           final_state=i if in_place else None)
        return _n(r.h), _n(r.final_state), _n(r.chunk_states)

    @staticmethod
    def gated_backward(x, gi, gr, lam, k, kind, cs, gh, gfinal=None, lengths=None, pad=0):
        n = None if lengths is None else torch.from_numpy(lengths).to(DEV)
        r = ssd.gated_scan_backward(_strided(x, kind, pad), _strided(gi, kind, pad), _strided(gr, kind, pad),
                                    _t(lam), _t(cs), _t(gh, kind), grad_final_state=_t(gfinal), decay_scale=k,
                                    lengths=n)
        return [_n(v) for v in r]

    @staticmethod
    def norm(x, res, w, eps, kind, y=True, fp8=True, pad=0, in_place=False):
        z = None if res is None else _t(res, kind) if in_place else _strided(res, kind, pad)
        r = ssd.rms_norm(_strided(x, kind, pad), _t(w), residual=z, eps=eps, want_y=y, fp8=fp8, want_rstd=True,
                         residual_out=z if in_place else None)
        return dict(y=_n(r.y), s=_n(r.residual), q=_n(r.q), scale=_n(r.scale), rstd=_n(r.rstd))

    @staticmethod
    def norm_backward(s, w, rstd, gy, gs, kind, pad=0):
        gx, gw = ssd.rms_norm_backward(_strided(s, kind, pad), _t(w), _t(rstd), _strided(gy, kind, pad),
                                       grad_residual=None if gs is None else _strided(gs, kind, pad))
        return _n(gx), _n(gw)

    @staticmethod
    def quantise(x, kind, block_rows, turn, pad=0, q_pad=0):
        R, C = x.shape[::-1] if turn else x.shape
        flat = torch.full((R, C + q_pad), 0xff, dtype=torch.uint8, device=DEV)
        q, scale = ssd.fp8_quantise(_strided(x, kind, pad), block_rows=block_rows, transpose=turn,
                                    q=flat.view(FP8)[:, :C])
        assert (flat[:, C:] == 0xff).all()
        return flat[:, :C].cpu().numpy(), _n(scale)

    @staticmethod
    def matmul(a, sa, b, sb, block_rows, out, a_pad=0, b_pad=0, out_pad=0, align=16):
        o = torch.full((a.shape[0], b.shape[0] + out_pad), -77.0, dtype=KIND[out], device=DEV)
        ssd.fp8_matmul(_fp8(a, a_pad, align), _t(sa), _fp8(b, b_pad, align), _t(sb), block_rows=block_rows,
                       out_dtype=KIND[out], out=o[:, :b.shape[0]])
        assert (o[:, b.shape[0]:] == -77.0).all()
        return _n(o[:, :b.shape[0]])


@pytest.mark.parametrize("case", cases.GATED, ids=str)
def test_gated_scan(case):
    cases.gated(_Gpu, *case)


@pytest.mark.parametrize("case", cases.GATED, ids=str)
def test_gated_scan_backward(case):
    cases.gated_backward(_Gpu, *case)


@pytest.mark.parametrize("case", cases.NORM, ids=str)
def test_rms_norm(case):
    cases.norm(_Gpu, *case)


@pytest.mark.parametrize("case", cases.NORM, ids=str)
def test_rms_norm_backward(case):
    cases.norm_backward(_Gpu, *case)


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("case", cases.QUANTISE, ids=str)
def test_fp8_quantise(case, block_rows, turn):
    cases.quantise(_Gpu, *case, block_rows, turn)


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_fp8_quantise_infinite(block_rows, turn):
    cases.quantise_special(_Gpu, block_rows, turn)


@pytest.mark.parametrize("align", [16, 1])
@pytest.mark.parametrize("case", cases.MATMUL, ids=str)
def test_fp8_matmul(case, align):
    cases.matmul(_Gpu, *case, align=align)


def test_gated_lengths_and_empty_rows():
    cases.gated_lengths_clamped(_Gpu)
    cases.gated_empty_row_infinite(_Gpu)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 70, 300])
def test_fp8_matmul_nan(M, out):
    cases.matmul_special(_Gpu, M, out)


def test_refusals_on_the_device():
    x = torch.zeros(2, 6, 8, device=DEV)
    lam = torch.zeros(8, device=DEV)
    neg = torch.complex(x, x).conj().imag           # a lazily negated view
    for bad in (x.half(), x.cpu(), x[0], neg, x[..., :4], x.transpose(0, 1), x[:1].expand(2, 6, 8)):
        with pytest.raises(ValueError):
            ssd.gated_scan(x, bad, x, lam)
        with pytest.raises(ValueError):
            ssd.rms_norm(x, lam, residual=bad)
    for kw in (dict(lengths=torch.zeros(2, device=DEV)), dict(lengths=torch.zeros(3, dtype=torch.int32, device=DEV)),
               dict(initial_state=torch.zeros(2, 7, device=DEV)), dict(h=torch.zeros(2, 6, 16, device=DEV)[..., ::2])):
        with pytest.raises(ValueError):
            ssd.gated_scan(x, x, x, lam, **kw)
    with pytest.raises(ssd.SSDError):
        ssd.gated_scan(x, x, x, lam, h=x)
    with pytest.raises(ssd.SSDError):
        ssd.rms_norm(x, lam, want_y=False)
    with pytest.raises(ssd.SSDError):
        ssd.rms_norm(torch.zeros(2, 16385, device=DEV), torch.zeros(16385, device=DEV))
    q, s = ssd.fp8_quantise(x)
    for a, sa, b, sb in ((q, s, q, s), (q, s[:, :5], q[0], s[:, :6]), (q.view(torch.uint8), s, q[0], s)):
        with pytest.raises(ValueError):
            ssd.fp8_matmul(a, sa, b, sb, block_rows=1)
    with pytest.raises(ValueError):
        ssd.fp8_matmul(q, s, q[0], s[:, :6].contiguous(), block_rows=1, out_dtype=torch.float16)


def test_rows_past_32_bit_offsets():
    """Column ranges of matrices of more than 2^32 elements, against the same values packed."""
    S, C = 65536, 100
    rows = 2 ** 32 // S + 64
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))  # noqa: E731
    wide = torch.empty(rows, S, dtype=torch.bfloat16, device=DEV)[:, S - C:]
    wide.copy_(torch.randn(rows, C, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    dense = wide.contiguous()
    w = torch.linspace(0.5, 2, C, device=DEV)
    a, b = (ssd.rms_norm(v, w, residual=v, want_rstd=True) for v in (wide, dense))
    assert same(a.y, b.y) and same(a.residual, b.residual)
    a, b = (ssd.rms_norm_backward(v, w, a.rstd, v, grad_residual=v) for v in (wide, dense))
    assert same(a[0], b[0]) and same(a[1], b[1])
    lam = torch.linspace(-9, 0, C, device=DEV)
    wide, dense = wide[None], dense[None]
    a, b = (ssd.gated_scan(v, v, v, lam, want_chunk_states=True) for v in (wide, dense))
    assert all(same(p, q) for p, q in zip(a, b))
    a, b = (ssd.gated_scan_backward(v, v, v, lam, a.chunk_states, dense) for v in (wide, dense))
    assert all(same(p, q) for p, q in zip(a, b))
    wide, dense = wide[0], dense[0]
    for turn in (False, True):
        a, b = (ssd.fp8_quantise(v, transpose=turn) for v in (wide, dense))
        assert same(a[0].contiguous(), b[0]) and same(a[1], b[1])
    q, s = ssd.fp8_quantise(dense)
    del wide
    far = torch.empty(rows, S, dtype=torch.uint8, device=DEV)[:, S - 112:S - 12].view(FP8)
    far.view(torch.uint8).copy_(q.view(torch.uint8))
    assert far.data_ptr() % 16 == 0
    qb, sb = ssd.fp8_quantise(torch.randn(64, C, device=DEV), block_rows=128)
    out = torch.empty(rows, S, dtype=torch.bfloat16, device=DEV)[:, S - 64:]
    ssd.fp8_matmul(far, s, qb, sb, out=out)
    assert same(out.contiguous(), ssd.fp8_matmul(q, s, qb, sb))


# ------------------------------------------------------------------- calls as a program makes them

def _calls(seed, T=700):
    """Every operator once on inputs from `seed`: inputs (dict of tensors) and a function of
    them that returns a list of outputs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    t = dict(rows=r(2, T, 3 * 96).to(torch.bfloat16), lam=-4 + r(96), init=r(2, 96),
             x=r(300, 1024).to(torch.bfloat16), res=r(300, 1024).to(torch.bfloat16), w=1 + 0.1 * r(1024),
             W=r(640, 1024) / 32, gh=r(2, T, 96).to(torch.bfloat16))

    def call(t):
        x, gi, gr = t["rows"].chunk(3, 2)
        s = ssd.gated_scan(x, gi, gr, t["lam"], initial_state=t["init"], want_chunk_states=True)
        b = ssd.gated_scan_backward(x, gi, gr, t["lam"], s.chunk_states, t["gh"])
        n = ssd.rms_norm(t["x"], t["w"], residual=t["res"], fp8=True, want_rstd=True)
        nb = ssd.rms_norm_backward(n.residual, t["w"], n.rstd, t["res"], grad_residual=t["x"])
        W, Ws = ssd.fp8_quantise(t["W"], block_rows=128)
        y = ssd.fp8_matmul(n.q, n.scale, W, Ws)
        yt, yts = ssd.fp8_quantise(y, transpose=True)
        xt, xts = ssd.fp8_quantise(n.y, transpose=True)
        gw = ssd.fp8_matmul(yt, yts, xt, xts, block_rows=1, out_dtype=torch.float32)
        return [*s, *b, n.y, n.residual, n.scale, n.q.view(torch.uint8), n.rstd, *nb, y, gw]
    return t, call


def _same(a, b):
    """"" where all outputs are equal, else which ones are not."""
    return " ".join(str(k) for k, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y))


def test_captured_calls_replay():
    t, call = _calls(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(t)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(t)
    torch.cuda.synchronize()
    for seed in (2, 3, 4):
        new, _ = _calls(seed)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, call(new)) == "", seed
        torch.cuda.synchronize()


def test_two_graphs_run_side_by_side():
    graphs = []
    for seed in (5, 6):
        t, call = _calls(seed)
        call(t)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(t)
        graphs.append((graph, out, call(t), t))  # the inputs live as long as the graph
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (graph, _, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in graphs:
            assert _same(out, want) == ""


def test_another_stream_and_repeated_calls():
    t, call = _calls(7)
    want = call(t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        with torch.cuda.stream(side):
            got = call(t)
        side.synchronize()
        assert _same(got, want) == ""


def test_steps_of_one_token_follow_the_scan():
    """Tokens one at a time, the state in place, against the whole sequence at once."""
    B, T, C = 3, 40, 70
    x, gi, gr, lam, init, _ = ref.gated_case(B, T, C, "f32", 11, state=True)
    want, err = ref.gated(x, gi, gr, lam, 8.0, init)
    state = _t(init)
    x, gi, gr, lam = (_t(v) for v in (x, gi, gr, lam))
    for t in range(T):
        h = ssd.gated_scan(x[:, t:t + 1], gi[:, t:t + 1], gr[:, t:t + 1], lam, initial_state=state,
                           final_state=state).h
        ref.close(_n(h)[:, 0], want[0][:, t], err[0][:, t], "f32", t)
    ref.close(_n(state), want[1], err[1], "f32", "final")


@pytest.mark.parametrize("B,T,C", [(2, 3000, 256), (300, 20, 64), (260, 32, 6), (260, 33, 6), (140, 600, 100)])
def test_gated_scan_in_bfloat16_of_many_groups(B, T, C):
    """Two channels per lane in segments, walks of more than eight tokens, a padded batch."""
    lengths = [T - (T // 2) * (b % 3 == 1) for b in range(B)]
    cases.gated(_Gpu, B, T, C, "bf16", True, lengths, 2)
    cases.gated_backward(_Gpu, B, T, C, "bf16", True, lengths, 2)


@pytest.mark.parametrize("B,T,C", [(32, 130, 256), (1, 9000, 320), (300, 70, 64), (300, 20, 64), (2, 4200, 3000), (8, 600, 1024)])
def test_gated_scan_of_many_groups(B, T, C):
    """Grids beyond the emulator's: many sequences, and a long one cut into many segments. Against
    torch in float64, one token after the other."""
    g = torch.Generator(device=DEV).manual_seed(B)
    x, gi, gr, gh = (torch.randn(B, T, C, generator=g, device=DEV).clamp(-6, 6) for _ in range(4))
    lam = torch.linspace(-9, 0, C, device=DEV)
    r = ssd.gated_scan(x, gi, gr, lam, want_chunk_states=True)
    b = ssd.gated_scan_backward(x, gi, gr, lam, r.chunk_states, gh)
    args = [v.double().cpu().numpy() for v in (x, gi, gr, lam)]
    want, err = ref.gated(*args, 8.0)
    for got, w, e in zip(r, (want[0], want[1], want[2]), err):
        ref.close(_n(got), w, e, "f32")
    want, err = ref.gated_backward(*args, 8.0, np.zeros((B, C)), gh.double().cpu().numpy())
    for got, w, e in zip(b, want, err):
        ref.close(_n(got), w, e, "f32")


@pytest.mark.parametrize("M,N,K,block_rows,out", [
    (1, 5136, 1024, 128, "bf16"), (33, 5136, 1024, 128, "bf16"), (64, 1024, 2048, 1, "f32"),
    (257, 1040, 1024, 128, "bf16"), (1000, 520, 1000, 128, "f32"), (2048, 1296, 640, 128, "bf16"),
    (5136, 1024, 1280, 1, "f32"), (640, 512, 20000, 1, "f32"), (4097, 5136, 256, 128, "bf16"), (515, 300, 8192, 128, "f32"),
    (5136, 2100, 256, 1, "f32"), (5136, 2100, 256, 128, "f32"), (4400, 5000, 200, 1, "bf16"), (2000, 9000, 1, 128, "bf16")])
def test_fp8_matmul_of_many_tiles(M, N, K, block_rows, out):
    cases.matmul(_Gpu, M, N, K, block_rows, out, -K % 16, -K % 16, 0)


@pytest.mark.parametrize("rows,F", [(3000, 1024), (9000, 200), (1500, 5000), (5000, 1024)])
def test_norm_of_many_rows(rows, F):
    cases.norm(_Gpu, rows, F, "bf16", True, 0)
    cases.norm_backward(_Gpu, rows, F, "bf16", True, 0)


def test_empty_calls():
    e = lambda *s, **k: torch.empty(*s, device=DEV, **k)  # noqa: E731
    r = ssd.gated_scan(e(0, 5, 4), e(0, 5, 4), e(0, 5, 4), e(4))
    assert r.h.shape == (0, 5, 4)
    init = torch.randn(2, 4, device=DEV)
    z = torch.zeros(2, 0, 4, device=DEV)
    r = ssd.gated_scan(z, z, z, e(4), initial_state=init, want_chunk_states=True)
    assert torch.equal(r.final_state, init)
    b = ssd.gated_scan_backward(z, z, z, e(4), r.chunk_states, z, grad_final_state=init)
    assert torch.equal(b.initial_state, init) and (b.lam == 0).all()
    assert ssd.rms_norm(e(0, 8), e(8), fp8=True).q.shape == (0, 8)
    gx, gw = ssd.rms_norm_backward(e(0, 8), e(8), e(0), e(0, 8))
    assert gx.shape == (0, 8) and (gw == 0).all()
    q, s = ssd.fp8_quantise(e(0, 8))
    assert q.shape == (0, 8)
    assert ssd.fp8_matmul(q, s, *ssd.fp8_quantise(torch.ones(3, 8, device=DEV), block_rows=128)).shape == (0, 3)
    none = torch.empty(2, 0, dtype=torch.uint8, device=DEV).view(FP8)
    assert (ssd.fp8_matmul(none, e(0, 2), none, e(1, 0)) == 0).all()


def test_together_with_the_scan():
    """One mixer block in 8 bits, as it would run: norm -> in_proj -> scan (bfloat16 rows) -> head
    mixer -> 8 bits -> out_proj, and a gated recurrence on projected rows; then the gradients of
    out_proj. Every product against float64 of the operands that it was given."""
    B, T, H, N, D = 2, 96, 4, 16, 32
    F, S = H * D, ssd.proj_width(H, N, D)
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, res = r(B, T, F).to(torch.bfloat16), r(B, T, F).to(torch.bfloat16)
    W_in, W_out, W_gate = r(S, F) / F ** 0.5, r(F, F) / F ** 0.5, r(3 * F, F) / F ** 0.5
    A = torch.complex(-0.05 - r(H).abs(), r(H))

    def product(q, qs, w, ws, block_rows, got, kind):
        b = lambda v: v.contiguous().view(torch.uint8).reshape(-1, v.shape[-1]).cpu().numpy()  # noqa: E731
        want, err = ref.matmul(ref.E4M3[b(q)], _n(qs), ref.E4M3[b(w)], _n(ws), block_rows, kind)
        ref.close(_n(got).reshape(want.shape), want, err, kind)

    n = ssd.rms_norm(x, torch.ones(F, device=DEV), residual=res, fp8=True)
    w_in, w_in_s = ssd.fp8_quantise(W_in, block_rows=128)
    rows = ssd.fp8_matmul(n.q, n.scale, w_in, w_in_s)
    product(n.q, n.scale, w_in, w_in_s, 128, rows, "bf16")
    y, _ = ssd.chunk_forward_proj(rows, A, H, N, D)
    same, _ = ssd.chunk_forward_proj(rows.float(), A, H, N, D)
    assert torch.equal(y, same)   # the scan widens bfloat16 rows
    z = ssd.head_mix(y, torch.eye(F, device=DEV)).view(B, T, F)
    q, qs = ssd.fp8_quantise(z)
    ref.check_quantised(_n(z).reshape(-1, F).astype(np.float64), 0.0, _n(q.contiguous()).reshape(-1, F), _n(qs).astype(np.float64), 1)
    w_out, w_out_s = ssd.fp8_quantise(W_out, block_rows=128)
    o = ssd.fp8_matmul(q, qs, w_out, w_out_s)
    product(q, qs, w_out, w_out_s, 128, o, "bf16")

    w_gate, w_gate_s = ssd.fp8_quantise(W_gate, block_rows=128)
    gate_rows = ssd.fp8_matmul(n.q, n.scale, w_gate, w_gate_s)
    gx, gi, gr = (v.clamp(-6, 6) for v in gate_rows.chunk(3, -1))
    lam = torch.full((F,), -4.0, device=DEV)
    h = ssd.gated_scan(*gate_rows.clamp(-6, 6).chunk(3, -1), lam).h
    want, err = ref.gated(*(v.double().cpu().numpy() for v in (gx, gi, gr, lam)), 8.0)
    ref.close(_n(h), want[0], err[0], "bf16")

    go = r(B, T, F).to(torch.bfloat16)
    gq, gqs = ssd.fp8_quantise(go)
    wt, wts = ssd.fp8_quantise(W_out, block_rows=128, transpose=True)
    assert torch.equal(wt.view(torch.uint8), w_out.view(torch.uint8).t()) and torch.equal(wts, w_out_s.t())
    product(gq, gqs, wt, wts, 128, ssd.fp8_matmul(gq, gqs, wt, wts), "bf16")
    gt, gts = ssd.fp8_quantise(go, transpose=True)
    zt, zts = ssd.fp8_quantise(z, transpose=True)
    product(gt, gts, zt, zts, 1, ssd.fp8_matmul(gt, gts, zt, zts, block_rows=1, out_dtype=torch.float32), "f32")
