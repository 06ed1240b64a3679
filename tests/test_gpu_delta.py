"""The gated delta rule on the GPU, through the Python entry points: the emulator's cases against float64
formulas, then what only a GPU shows (captured and replayed calls, other streams, repeated calls bit for bit,
large sizes, offsets past 32 bits)."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import complex_chunkwise_ssd_amd as ssd
import delta_cases as cases
import delta_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


def _t(v, kind="f32"):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(KIND[kind]).to(DEV)


def _strided(v, kind, pad):
    """v (B, T, H, D) with its tokens `pad` elements further apart, NaN between them."""
    t = _t(v, kind)
    if not pad:
        return t
    B, T, H, D = t.shape
    wide = torch.full((B, T, H * D + pad), float("nan"), dtype=t.dtype, device=DEV)
    wide[..., :H * D] = t.flatten(2)
    return wide[..., :H * D].unflatten(-1, (H, D))


def _n(t):
    if t is None:
        return None
    torch.cuda.synchronize()
    return t.float().cpu().numpy()


def _lengths(n):
    return None if n is None else torch.from_numpy(np.asarray(n, np.int32)).to(DEV)


class _Gpu:
    """The functions of delta_emu_harness on the GPU."""

    @staticmethod
    def delta(q, k, v, g, beta, scale, kind, init=None, lengths=None, states=False, pad=0, in_place=False):
        i = _t(init)
        r = ssd.gated_delta(_strided(q, kind, pad), _strided(k, kind, pad), _strided(v, kind, pad), _t(g), _t(beta),
                            scale=scale, initial_state=i, lengths=_lengths(lengths), want_chunk_states=states,
                            final_state=i if in_place else None)
        return _n(r.o), _n(r.final_state), _n(r.chunk_states)

    @staticmethod
    def delta_backward(q, k, v, g, beta, scale, kind, states, go, gfinal=None, lengths=None, pad=0):
        r = ssd.gated_delta_backward(_strided(q, kind, pad), _strided(k, kind, pad), _strided(v, kind, pad), _t(g),
                                     _t(beta), _t(states), _t(go, kind), grad_final_state=_t(gfinal), scale=scale,
                                     lengths=_lengths(lengths))
        return [_n(v) for v in r]


@pytest.mark.parametrize("case", cases.DELTA, ids=str)
def test_gated_delta(case):
    cases.forward(_Gpu, *case)


@pytest.mark.parametrize("case", cases.DELTA, ids=str)
def test_gated_delta_backward(case):
    cases.backward(_Gpu, *case)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_same_keys(kind):
    cases.same_keys(_Gpu, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_columns_apart(kind):
    cases.columns_apart(_Gpu, kind)


def test_lengths_and_decays_clamped():
    cases.clamped(_Gpu)


def test_empty_row_infinite():
    cases.empty_row_infinite(_Gpu)


def _inputs(B, T, Hk, Hv, Dk, Dv, kind, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(B, T, Hk, Dk), dim=-1).to(KIND[kind]) for _ in range(2))
    v = r(B, T, Hv, Dv).to(KIND[kind])
    decay = -torch.exp(torch.rand(B, T, Hv, generator=g, device=DEV) * 5 - 6)
    return q, k, v, decay, torch.sigmoid(r(B, T, Hv)), r(B, Hv, Dk, Dv) * 0.3


def _both(args, init, go, lengths=None):
    r = ssd.gated_delta(*args, initial_state=init, lengths=lengths, want_chunk_states=True)
    return list(r) + list(ssd.gated_delta_backward(*args, r.chunk_states, go, grad_final_state=init, lengths=lengths))


@pytest.mark.parametrize("sizes", [(2, 300, 2, 4, 64, 64, "bf16"), (3, 130, 1, 2, 100, 40, "f32"), (4, 3, 2, 2, 64, 128, "bf16")])
def test_repeated_calls_give_the_same_bits(sizes):
    *args, init = _inputs(*sizes)
    go = torch.randn_like(args[2].float()).to(args[2].dtype)
    first = [t.clone() for t in _both(args, init, go)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(_both(args, init, go), first))


@pytest.mark.parametrize("sizes", [(2, 300, 2, 4, 64, 64, "bf16"), (5, 1, 2, 4, 64, 64, "bf16")])
def test_captured_and_replayed(sizes):
    """Replays with new inputs, eager work and synchronisation between them, against eager calls."""
    *args, init = _inputs(*sizes)
    go = torch.randn_like(args[2].float()).to(args[2].dtype)
    _both(args, init, go)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _both(args, init, go)
    for seed in (1, 2, 3, 4):
        new = _inputs(*sizes, seed=seed)
        for a, b in zip(args + [init], new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = _both(args, init, go)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_on_another_stream():
    *args, init = _inputs(2, 200, 1, 2, 64, 64, "bf16")
    want = _both(args, init, args[2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _both(args, init, args[2])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_split_calls_continue_the_state(kind):
    """A sequence in several calls, each from the one before's final state, token by token at the end."""
    q, k, v, g, beta, init = _inputs(2, 200, 1, 2, 64, 48, kind)
    whole = ssd.gated_delta(q, k, v, g, beta, initial_state=init)
    at, state, o = 0, init.clone(), []
    for step in (128, 64, 5, 1, 1, 1):
        part = [w[:, at:at + step].contiguous() for w in (q, k, v, g, beta)]
        r = ssd.gated_delta(*part, initial_state=state, final_state=state)
        o.append(r.o)
        at += step
    assert at == 200
    o = torch.cat(o, 1).float()
    # the same sums in another order: 64 units of their size (delta_ref.close), and two roundings of o
    size = whole.o.float().square().mean().sqrt()
    assert (o - whole.o.float()).square().mean().sqrt() <= (64 * ref.U + 2 * ref.HALF[kind]) * size
    assert (state - whole.final_state).norm() <= 128 * ref.U * state.norm()


def test_column_ranges_of_projected_rows():
    q, k, v, g, beta, init = _inputs(2, 100, 2, 4, 64, 32, "bf16")
    rows = torch.full((2, 100, 2 * 128 + 128 + 3), float("nan"), dtype=torch.bfloat16, device=DEV)
    parts = []
    at = 3
    for w in (q, k, v):
        n = w[0, 0].numel()
        rows[..., at:at + n] = w.flatten(2)
        parts.append(rows[..., at:at + n].unflatten(-1, w.shape[2:]))
        at += n
    a = _both([q, k, v, g, beta], init, v)
    b = _both([*parts, g, beta], init, v)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("sizes", [(32, 2048, 16, 16, 64, 64, "bf16"), (3, 5000, 2, 4, 128, 128, "bf16"), (2, 1000, 3, 6, 72, 100, "f32")])
def test_large_against_tokens_in_float64(sizes):
    """The value heads of one key head of the last row of a large call against the definition, outputs and
    gradients."""
    q, k, v, g, beta, init = _inputs(*sizes)
    kind = sizes[-1]
    B, T, Hv = g.shape
    lengths = torch.full((B,), T, dtype=torch.int32, device=DEV)
    lengths[B - 1] = T - 77
    go = torch.randn_like(v.float()).to(v.dtype)
    got = _both([q, k, v, g, beta], init, go, lengths)
    share = Hv // q.shape[2]
    b, h = B - 1, slice(0, share)
    pick = [w[b:b + 1, :, :1] for w in (q, k)] + [w[b:b + 1, :, h] for w in (v, g, beta)]
    pick = [w.double().cpu().numpy() for w in pick]
    i0 = init[b:b + 1, h].double().cpu().numpy()
    n, scale = np.array([T - 77]), float(np.float32(q.shape[3]) ** np.float32(-0.5))
    o, final, states = ref.tokens(*pick, scale, i0, n)
    grads = ref.tokens_backward(*pick, scale, i0, go[b:b + 1, :, h].double().cpu().numpy(), i0, n)
    mine = [got[0][b:b + 1, :, h], got[1][b:b + 1, h], got[2][b:b + 1, :, h], got[3][b:b + 1, :, :1], got[4][b:b + 1, :, :1],
            got[5][b:b + 1, :, h], got[6][b:b + 1, :, h], got[7][b:b + 1, :, h], got[8][b:b + 1, h]]
    # errors of random sign do not grow along the sequence (the map is a contraction): 64 units of
    # rounding of the whole (delta_ref.close), and the results' own
    for i, (x, y) in enumerate(zip(mine, [o, final, states] + grads)):
        x = x.double().cpu().numpy()
        off = np.sqrt(((x - y) ** 2).sum() / (y ** 2).sum())
        half = ref.HALF[kind] if i in (0, 3, 4, 5) else 0.0
        print(i, off)
        assert off <= 64 * ref.U + half, (i, off)


def test_offsets_past_32_bits():
    """A state of 4.3 GiB (the last row's offset passes 2^32 bytes), chunk and step."""
    B, Hv, D = 4097, 16, 128
    init = torch.zeros(B, Hv, D, D, device=DEV)
    q, k, v, g, beta, small = _inputs(1, 20, 16, 16, D, D, "bf16")
    init[-1] = small[0]
    for T in (1, 20):
        want = ssd.gated_delta(*[w[:, :T].contiguous() for w in (q, k, v, g, beta)], initial_state=small)
        args = [w[:, :T].expand(B, *w[:, :T].shape[1:]).contiguous() for w in (q, k, v, g, beta)]
        got = ssd.gated_delta(*args, initial_state=init)
        assert torch.equal(got.o[-1], want.o[0]) and torch.equal(got.final_state[-1], want.final_state[0])
        del got, args
