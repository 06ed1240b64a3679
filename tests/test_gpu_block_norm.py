"""The norms around a block on the GPU, through the Python entry points: the emulator's cases against float64
formulas, then what only a GPU shows, and a run of the operators of a delta-rule block together."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import block_norm_cases as cases
import complex_chunkwise_ssd_amd as ssd
import delta_ref
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


class _Gpu:
    """The functions of block_norm_harness on the GPU."""

    @staticmethod
    def gated_norm(x, z, w, eps, kind, y=True, fp8=True, pad=0):
        r = ssd.gated_norm(_strided(x, kind, pad), _strided(z, kind, pad), _t(w), eps=eps, want_y=y, fp8=fp8,
                           want_rstd=True)
        return dict(y=_n(r.y), q=_n(r.q), scale=_n(r.scale), rstd=_n(r.rstd))

    @staticmethod
    def gated_norm_backward(x, z, w, rstd, gy, kind, pad=0):
        return [_n(v) for v in ssd.gated_norm_backward(_strided(x, kind, pad), _strided(z, kind, pad), _t(w), _t(rstd),
                                                       _strided(gy, kind, pad))]

    @staticmethod
    def block_norm(x, res, w1, w2, alpha, eps, kind, y=True, fp8=True, pad=0, in_place=False):
        z = _t(res, kind) if in_place else _strided(res, kind, pad)
        r = ssd.block_norm(_strided(x, kind, pad), z, _t(w1), _t(w2), residual_scale=alpha, eps=eps, want_y=y, fp8=fp8,
                           want_rstd=True, residual_out=z if in_place else None)
        return dict(y=_n(r.y), s=_n(r.residual), q=_n(r.q), scale=_n(r.scale), post=_n(r.post_rstd), pre=_n(r.pre_rstd))

    @staticmethod
    def block_norm_backward(x, s, w1, w2, r1, r2, alpha, gy, gs, kind, pad=0):
        return [_n(v) for v in ssd.block_norm_backward(
            _strided(x, kind, pad), _strided(s, kind, pad), _t(w1), _t(w2), _t(r1), _t(r2), _strided(gy, kind, pad),
            grad_residual=None if gs is None else _strided(gs, kind, pad), residual_scale=alpha)]


@pytest.mark.parametrize("case", cases.GATED, ids=str)
def test_gated_norm(case):
    cases.run_gated(_Gpu, *case)


@pytest.mark.parametrize("case", cases.GATED, ids=str)
def test_gated_norm_backward(case):
    cases.run_gated_backward(_Gpu, *case)


@pytest.mark.parametrize("case", cases.BLOCK, ids=str)
def test_block_norm(case):
    cases.run_block(_Gpu, *case)


@pytest.mark.parametrize("case", cases.BLOCK, ids=str)
def test_block_norm_backward(case):
    cases.run_block_backward(_Gpu, *case)


def test_rows_apart():
    cases.rows_apart(_Gpu)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def _both(x, z, gy, w, w2):
    a = ssd.gated_norm(x, z, w, fp8=True, want_rstd=True)
    b = ssd.block_norm(x, z, w2, w2, residual_scale=0.5, fp8=True, want_rstd=True)
    return [*a, *ssd.gated_norm_backward(x, z, w, a.rstd, gy), *b,
            *ssd.block_norm_backward(x, b.residual, w2, w2, b.post_rstd, b.pre_rstd, gy, grad_residual=gy, residual_scale=0.5)]


def _same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


@pytest.mark.parametrize("H,D", [(16, 64), (10, 100)])
def test_repeated_captured_and_on_another_stream(H, D):
    F = H * D
    make = lambda seed: [_randn(seed + i, 5000, F).to(torch.bfloat16) for i in range(3)]  # noqa: E731
    args, w, w2 = make(1), 1 + 0.1 * _randn(8, D), 1 + 0.1 * _randn(9, F)
    first = _both(*args, w, w2)
    for _ in range(3):
        assert _same(_both(*args, w, w2), first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _both(*args, w, w2)
    side.synchronize()
    assert _same(got, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _both(*args, w, w2)
    for seed in (10, 20, 30):
        for a, b in zip(args, make(seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = _both(*args, w, w2)
        torch.cuda.synchronize()
        assert _same(out, want), seed


def test_many_rows_against_float64():
    """More rows than workgroups hold: each row as it is alone, the weights' gradients against float64."""
    x, z, gy = (_randn(i, 40000, 320).to(torch.bfloat16) for i in range(3))
    w, w2 = 1 + 0.1 * _randn(8, 40), 1 + 0.1 * _randn(9, 320)
    all_rows = _both(x, z, gy, w, w2)
    at = slice(39990, 40000)
    few = _both(x[at], z[at], gy[at], w, w2)
    for i in (0, 1, 3, 4, 5, 7, 8, 9, 11, 12, 13, 14):
        assert _same([all_rows[i][at]], [few[i]]), i
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, err = cases.gated_backward(d(x).clip(-6, 6), d(z).clip(-6, 6), d(w), d(all_rows[3]), d(gy))
    ref.close(_n(all_rows[6]), want[2], err[2], "f32", "weight")
    want, err = cases.block_backward(d(x), d(all_rows[8]), d(w2), d(w2), d(all_rows[11]), d(all_rows[12]), 0.5, d(gy), d(gy))
    ref.close(_n(all_rows[15]), want[2], err[2], "f32", "post_weight")
    ref.close(_n(all_rows[16]), want[3], err[3], "f32", "pre_weight")


def test_rows_past_32_bit_offsets():
    """Column ranges of matrices of more than 2^32 elements, against the same values packed."""
    S, F = 65536, 160
    rows = 2 ** 32 // S + 64
    wide = torch.empty(rows, S, dtype=torch.bfloat16, device=DEV)[:, S - F:]
    wide.copy_(_randn(1, rows, F))
    dense, w, w2 = wide.contiguous(), 1 + 0.1 * _randn(8, 20), 1 + 0.1 * _randn(9, F)
    assert _same(_both(wide, wide, wide, w, w2), _both(dense, dense, dense, w, w2))


def test_refusals_on_the_device():
    x, w, w8 = torch.zeros(2, 6, 32, device=DEV), torch.zeros(32, device=DEV), torch.zeros(8, device=DEV)
    for bad in (x.half(), x.cpu(), x[0], x[..., :4], x.transpose(0, 1), x[:1].expand(2, 6, 32)):
        with pytest.raises(ValueError):
            ssd.gated_norm(x, bad, w8)
        with pytest.raises(ValueError):
            ssd.block_norm(x, bad, w, w)
    for bad in (torch.zeros(7, device=DEV), torch.zeros(2, 8, device=DEV), w8.double(), w8.cpu()):
        with pytest.raises(ValueError):
            ssd.gated_norm(x, x, bad)
    for refused in (lambda: ssd.gated_norm(x, x, torch.zeros(4, device=DEV)), lambda: ssd.gated_norm(x, x, w8, y=x),
                    lambda: ssd.gated_norm(x, x, w8, want_y=False), lambda: ssd.block_norm(x, x, w, w, residual_out=x),
                    lambda: ssd.block_norm(x, x.clone(), w, w, want_y=False)):
        with pytest.raises(ssd.SSDError):
            refused()
    q = torch.zeros(2, 4, 2, 8, device=DEV)
    g = torch.zeros(2, 4, 2, device=DEV)
    for bad in (q.half(), q.cpu(), q[0], q[:, :3], q.transpose(0, 1), q.transpose(1, 2), q[:, :, :1].expand(2, 4, 2, 8)):
        with pytest.raises(ValueError):
            ssd.gated_delta(q, bad, q, g, g)
    for kw in (dict(lengths=torch.zeros(2, device=DEV)), dict(initial_state=torch.zeros(2, 2, 8, 7, device=DEV)),
               dict(o=torch.zeros(2, 4, 2, 16, device=DEV)[..., ::2])):
        with pytest.raises(ValueError):
            ssd.gated_delta(q, q, q, g, g, **kw)
    with pytest.raises(ValueError):
        ssd.gated_delta(q, q, q, g.bfloat16(), g)
    for refused in (lambda: ssd.gated_delta(q, q, q, g, g, o=q), lambda: ssd.gated_delta(q, q, q, g, g, scale=float("nan")),
                    lambda: ssd.gated_delta(q[:, :, :1].contiguous().expand(2, 4, 1, 8).repeat(1, 1, 3, 1),
                                            q.repeat(1, 1, 2, 1)[:, :, :3].contiguous(), q, g, g)):
        with pytest.raises(ssd.SSDError):
            refused()


def test_nothing_to_do():
    x, w = torch.zeros(0, 32, device=DEV), torch.ones(32, device=DEV)
    assert ssd.gated_norm(x, x, w[:8].contiguous()).y.shape == (0, 32)
    g = ssd.gated_norm_backward(x, x, w[:8].contiguous(), torch.zeros(0, 4, device=DEV), x)
    assert g.x.shape == (0, 32) and (g.weight == 0).all()
    e = torch.zeros(0, device=DEV)
    g = ssd.block_norm_backward(x, x, w, w, e, e, x)
    assert (g.post_weight == 0).all() and (g.pre_weight == 0).all()
    q, state = torch.zeros(2, 0, 1, 8, device=DEV), torch.rand(2, 1, 8, 8, device=DEV)
    r = ssd.gated_delta(q, q, q, q[..., 0].contiguous(), q[..., 0].contiguous(), initial_state=state)
    assert torch.equal(r.final_state, state) and r.o.shape == (2, 0, 1, 8)
    assert (ssd.gated_delta(q, q, q, q[..., 0].contiguous(), q[..., 0].contiguous()).final_state == 0).all()
    b = ssd.gated_delta_backward(q, q, q, q[..., 0].contiguous(), q[..., 0].contiguous(),
                                 torch.zeros(2, 0, 1, 8, 8, device=DEV), q, grad_final_state=state)
    assert torch.equal(b.initial_state, state)


def test_a_delta_block_together():
    """A block as it would run: norm to 8 bits -> in_proj -> keys and queries scaled -> delta rule -> gated norm to
    8 bits -> out_proj -> the block's end and the next one's norm; then the gradients of everything but the
    products, each step against float64 of the operands that it was given. The second half of the sequence
    once more token by token from the first half's state."""
    B, T, Hk, Hv, D = 2, 96, 2, 4, 64
    F, K = Hv * D, Hk * D
    S = 2 * K + 2 * F
    x, res = _randn(1, B, T, F).to(torch.bfloat16), _randn(2, B, T, F).to(torch.bfloat16)
    ones = torch.ones(F, device=DEV)
    w_in, w_in_s = ssd.fp8_quantise(_randn(3, S, F) / F ** 0.5, block_rows=128)
    w_out, w_out_s = ssd.fp8_quantise(_randn(4, F, F) / F ** 0.5, block_rows=128)
    decay, beta = -torch.rand(B, T, Hv, device=DEV), torch.rand(B, T, Hv, device=DEV)
    b0 = ssd.block_norm(x, res, ones, ones, residual_scale=0.5, fp8=True, want_y=False)
    rows = ssd.fp8_matmul(b0.q, b0.scale, w_in, w_in_s)
    q, k, v, z = rows.split([K, K, F, F], -1)
    unit = torch.full((D,), D ** -0.5, device=DEV)
    heads = lambda t, h: t.unflatten(-1, (h, D))  # noqa: E731
    q, k = (ssd.rms_norm(heads(w.contiguous(), Hk), unit).y for w in (q, k))
    assert ((k.float() ** 2).sum(-1) - 1).abs().max() < 2 ** -6
    v = heads(v, Hv)
    r = ssd.gated_delta(q, k, v, decay, beta, want_chunk_states=True)
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    want = delta_ref.forward(d(q), d(k), d(v), d(decay), d(beta), D ** -0.5, None, None, "bf16")
    delta_ref.close(_n(r.o), want[0], "bf16", "o")
    delta_ref.close(_n(r.final_state), want[1], "f32", "final")
    w = 1 + 0.1 * _randn(5, D)
    n = ssd.gated_norm(r.o.flatten(-2), z, w, fp8=True, want_rstd=True)
    (y, _), (ey, _) = cases.gated(d(r.o).reshape(-1, F), d(z).reshape(-1, F).clip(-6, 6), d(w), D, 1e-6)
    assert float(z.abs().max()) <= 6
    ref.close(_n(n.y).reshape(-1, F), y, ey, "bf16", "gated")
    ref.check_quantised(y, ey, _n(n.q).reshape(-1, F), _n(n.scale).astype(np.float64), 1)
    out = ssd.fp8_matmul(n.q, n.scale, w_out, w_out_s)
    b1 = ssd.block_norm(out, b0.residual, ones, ones, residual_scale=0.5, want_rstd=True)
    (y, s, _, _), (ey, es, _, _) = cases.block(d(out).reshape(-1, F), d(b0.residual).reshape(-1, F), d(ones), d(ones), 0.5, 1e-6)
    ref.close(_n(b1.y).reshape(-1, F), y, ey, "bf16", "y")
    ref.close(_n(b1.residual).reshape(-1, F), s, es, "bf16", "s")

    # tokens 48 .. 95 one by one, on the state that the first 48 left
    half = [t[:, :48].contiguous() for t in (q, k, v, decay, beta)]
    state = ssd.gated_delta(*half).final_state
    steps = []
    for t in range(48, T):
        steps.append(ssd.gated_delta(*[a[:, t:t + 1].contiguous() for a in (q, k, v, decay, beta)], initial_state=state,
                                     final_state=state).o)
    late = torch.cat(steps, 1)
    bar = want[0].e[:, 48:] + 2.0 ** -8 * np.abs(want[0].v[:, 48:])
    assert (np.abs(_n(late) - want[0].v[:, 48:]) <= 1.01 * bar + 1e-6).all()

    gy, gs = _randn(6, B, T, F).to(torch.bfloat16), _randn(7, B, T, F).to(torch.bfloat16)
    gb = ssd.block_norm_backward(out, b1.residual, ones, ones, b1.post_rstd, b1.pre_rstd, gy, grad_residual=gs,
                                 residual_scale=0.5)
    flat = lambda t: d(t).reshape(-1, t.shape[-1])  # noqa: E731
    wantb, errb = cases.block_backward(flat(out), flat(b1.residual), d(ones), d(ones), d(b1.post_rstd), d(b1.pre_rstd), 0.5,
                                       flat(gy), flat(gs))
    for i, kind in enumerate(("bf16", "bf16", "f32", "f32")):
        ref.close(_n(gb[i]).reshape(wantb[i].shape), wantb[i], errb[i], kind, i)
    gn = ssd.gated_norm_backward(r.o.flatten(-2), z, w, n.rstd, gb.x)
    wantn, errn = cases.gated_backward(flat(r.o.flatten(-2)), flat(z), d(w), d(n.rstd), flat(gb.x))
    for i, kind in enumerate(("bf16", "bf16", "f32")):
        ref.close(_n(gn[i]).reshape(wantn[i].shape), wantn[i], errn[i], kind, i)
    go = gn.x.unflatten(-1, (Hv, D))
    gd = ssd.gated_delta_backward(q, k, v, decay, beta, r.chunk_states, go)
    wantd = delta_ref.backward(d(q), d(k), d(v), d(decay), d(beta), D ** -0.5, d(r.chunk_states), d(go), None, None)
    for i, kind in enumerate(("bf16", "bf16", "bf16", "f32", "f32", "f32")):
        delta_ref.close(_n(gd[i]), wantd[i], kind, i)
