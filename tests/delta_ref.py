"""The gated delta rule in float64 (test-only): one token after the other, with its gradients, and the
chunked form with bounds of what float32 arithmetic can make of it.

Bounds. A number carries the largest error that it can have; a product of matrices
X Y errs by |X| dY + dX |Y| and, computed as sums of n products in float32 from operands in 24 bits, by
(n + 64) 2 U |X| |Y| more: each of the n products and sums rounds once, the parts that are left out of an
operand are 2^-24 of it, and the joins of partial sums (up to eight levels of six parts) stay below 64. A
decay exp(d) is off by (|d| + 4) U of itself, at most 28 U where it counts (it is
below 2^-24 from |d| = 24 on). The state's error goes from chunk to chunk by the chunk's own map, whose
norm is at most 1 for keys of length 1: per column, e' = |M| e + what the chunk adds."""

import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
CHUNK = 64
TINY = 1e-30


def case(B, T, Hk, Hv, Dk, Dv, kind, seed, state=True, lengths=None, forget=False):
    """Inputs as the rule meets them: keys and queries of length 1 (as far as the type holds it)."""
    g = np.random.default_rng(seed)
    unit = lambda w: w / np.sqrt((w * w).sum(-1, keepdims=True))  # noqa: E731
    q, k = (rounded(unit(g.standard_normal((B, T, Hk, Dk)) + 0.3), kind) for _ in range(2))
    v = rounded(g.standard_normal((B, T, Hv, Dv)), kind)
    decay = -np.exp(g.uniform(np.log(1e-3), np.log(2.0), (B, T, Hv)))
    if forget:
        decay[g.random((B, T, Hv)) < 0.05] = -300.0
    decay = np.float32(decay).astype(np.float64)
    beta = np.float32(1 / (1 + np.exp(-2 * g.standard_normal((B, T, Hv))))).astype(np.float64)
    init = np.float32(0.3 * g.standard_normal((B, Hv, Dk, Dv))).astype(np.float64) if state else None
    n = None if lengths is None else np.asarray(lengths, np.int32)
    return q, k, v, decay, beta, init, n


def rounded(v, kind):
    v = np.asarray(v, np.float32)
    if kind == "bf16":
        u = v.view(np.uint32)
        v = ((u + 0x7fff + (u >> 16 & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)
    return v.astype(np.float64)


def tokens(q, k, v, g, beta, scale, init=None, lengths=None):
    """(o, final, states entering each chunk), from the definition."""
    B, T, Hv, Dv = v.shape
    share, Dk = Hv // q.shape[2], q.shape[3]
    S = np.zeros((B, Hv, Dk, Dv)) if init is None else init.copy()
    o, states = np.zeros(v.shape), np.zeros((B, -(-T // CHUNK), Hv, Dk, Dv))
    for t in range(T):
        if t % CHUNK == 0:
            states[:, t // CHUNK] = S
        qt, kt = (np.repeat(w[:, t], share, 1) for w in (q, k))
        live = np.ones(B, bool) if lengths is None else t < lengths
        new = S * np.exp(g[:, t])[..., None, None]
        u = beta[:, t][..., None] * (v[:, t] - np.einsum("bhkv,bhk->bhv", new, kt))
        new = new + kt[..., None] * u[..., None, :]
        S = np.where(live[:, None, None, None], new, S)
        o[:, t] = np.where(live[:, None, None], scale * np.einsum("bhkv,bhk->bhv", new, qt), 0.0)
    return o, S, states


def tokens_backward(q, k, v, g, beta, scale, init, go, gfinal=None, lengths=None):
    """Gradients (q, k, v, g, beta, init), from the definition."""
    B, T, Hv, Dv = v.shape
    share, Dk = Hv // q.shape[2], q.shape[3]
    S = np.zeros((B, Hv, Dk, Dv)) if init is None else init.copy()
    seen = []
    qs, ks = (np.repeat(w, share, 2) for w in (q, k))
    for t in range(T):
        live = (np.ones(B, bool) if lengths is None else t < lengths)[:, None, None, None]
        D = S * np.exp(g[:, t])[..., None, None]
        p = np.einsum("bhkv,bhk->bhv", D, ks[:, t])
        u = beta[:, t][..., None] * (v[:, t] - p)
        new = D + ks[:, t][..., None] * u[..., None, :]
        seen.append((D, p, u, new, live))
        S = np.where(live, new, S)
    gs = np.zeros_like(S) if gfinal is None else gfinal.copy()
    out = [np.zeros(qs.shape), np.zeros(qs.shape), np.zeros(v.shape), np.zeros(g.shape), np.zeros(g.shape)]
    for t in range(T - 1, -1, -1):
        D, p, u, new, live = seen[t]
        row = live[..., 0]
        before = gs
        n = gs + scale * qs[:, t][..., None] * go[:, t][..., None, :]
        gu = np.einsum("bhkv,bhk->bhv", n, ks[:, t])
        w = -beta[:, t][..., None] * gu
        out[0][:, t] = np.where(row, scale * np.einsum("bhkv,bhv->bhk", new, go[:, t]), 0)
        out[1][:, t] = np.where(row, np.einsum("bhkv,bhv->bhk", n, u) + np.einsum("bhkv,bhv->bhk", D, w), 0)
        out[2][:, t] = np.where(row, -w, 0)
        out[4][:, t] = np.where(row[..., 0], (gu * (v[:, t] - p)).sum(-1), 0)
        n = n + ks[:, t][..., None] * w[..., None, :]
        out[3][:, t] = np.where(row[..., 0], (n * D).sum((-2, -1)), 0)
        gs = np.where(live, n * np.exp(g[:, t])[..., None, None], before)
    for i in range(2):
        out[i] = out[i].reshape(B, T, -1, share, Dk).sum(3)
    return out + [gs]


class Num:
    """Values with the largest errors that they can have."""

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, np.float64)
        self.e = np.broadcast_to(np.asarray(e, np.float64), self.v.shape)

    @staticmethod
    def of(x):
        return x if isinstance(x, Num) else Num(x)

    def __add__(self, o):
        o = Num.of(o)
        v = self.v + o.v
        return Num(v, self.e + o.e + U * np.abs(v))

    def __neg__(self):
        return Num(-self.v, self.e)

    def __sub__(self, o):
        return self + -Num.of(o)

    def __mul__(self, o):
        o = Num.of(o)
        v = self.v * o.v
        return Num(v, np.abs(self.v) * o.e + self.e * np.abs(o.v) + self.e * o.e + U * np.abs(v))

    def __matmul__(self, o):
        return self.product(o, 0.0)

    def product(self, o, more):
        """self @ o, its operands held to `more` of themselves."""
        o = Num.of(o)
        a, b = np.abs(self.v), np.abs(o.v)
        n = self.v.shape[-1]
        return Num(self.v @ o.v, a @ o.e + self.e @ b + self.e @ o.e + (2 * U * (n + 64) + more) * (a @ b))

    @property
    def T(self):
        return Num(np.swapaxes(self.v, -1, -2), np.swapaxes(self.e, -1, -2))

    def sum(self, axis):
        n = self.v.shape[axis]
        return Num(self.v.sum(axis), self.e.sum(axis) + 2 * U * (n + 16) * np.abs(self.v).sum(axis))


def _exp(d):
    """exp of exact differences, with the error of float32."""
    v = np.exp(np.minimum(d, 700.0))
    return Num(v, v * U * (np.minimum(np.abs(d) * 1.4427, 24) + 4) + TINY)


class _Chunk:
    """One chunk of one head: q, k (n, Dk), v (n, Dv), g, beta (n), all float64 and exact."""

    def __init__(self, q, k, v, g, beta, scale):
        n = len(g)
        sums = np.cumsum(np.maximum(g, -1000.0))
        low, strict = np.tri(n, dtype=bool), np.tri(n, k=-1, dtype=bool)
        D = _exp(sums[:, None] - sums[None, :])
        self.D = Num(np.where(low, D.v, 0), np.where(low, D.e, 0))
        Ds = Num(np.where(strict, D.v, 0), np.where(strict, D.e, 0))
        self.strict = Ds
        self.q, self.k, self.v, self.beta, self.scale = Num(q), Num(k), Num(v), Num(beta[:, None]), scale
        self.since, self.left = self._col(_exp(sums)), self._col(_exp(sums[-1] - sums))
        self.whole = _exp(sums[-1:])
        self.kk = self.k @ self.k.T
        self.A = self.beta * Ds * self.kk
        inverse = np.linalg.inv(np.eye(n) + self.A.v) if n else np.zeros((0, 0))
        inverse = np.where(low, inverse, 0)
        # (I + A) X = R by substitution, and by blocks: X errs by |T| times (the residual's rounding
        # (2 n + 128) U |A| |X|, twice for the blocks' own inverses, plus dA |X| + dR)
        self.inverse = inverse
        self.P = (self.q @ self.k.T) * self.D * scale

    @staticmethod
    def _col(x):
        return Num(x.v[:, None], x.e[:, None])

    def solve(self, R, turned=False):
        t, A = (self.inverse.T, self.A.T) if turned else (self.inverse, self.A)
        n = len(t)
        x = t @ R.v
        res = R.e + U * np.abs(R.v) + (4 * U * (n + 64) * np.abs(A.v) + A.e) @ np.abs(t) @ np.abs(R.v)
        return Num(x, np.abs(t) @ res)

    def read(self, S):
        return self.v - self.since * (self.k @ S)

    def u(self, S):
        return self.solve(self.beta * self.read(S))

    def map(self):
        """The state's own map through the chunk, (Dk, Dk)."""
        k, since, left, beta = self.k.v, self.since.v, self.left.v, self.beta.v
        return self.whole.v * np.eye(k.shape[1]) - (left * k).T @ self.inverse @ (beta * since * k)


def _spread(column_norms, rows):
    """An error of that 2-norm in each column, as a bound of every element."""
    return np.broadcast_to(column_norms[None, :], (rows, len(column_norms)))


def _each(B, T, Hv, lengths):
    for b in range(B):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        for h in range(Hv):
            yield b, h, n


def forward(q, k, v, g, beta, scale, init, lengths, kind):
    """Num of (o, final, states)."""
    B, T, Hv, Dv = v.shape
    share, Dk = Hv // q.shape[2], q.shape[3]
    chunks = -(-T // CHUNK)
    more = 2.0 ** -15 if kind == "bf16" else 0.0  # two parts of 8 bits in what only reaches o
    o, fin, st = (np.zeros((2,) + s) for s in (v.shape, (B, Hv, Dk, Dv), (B, chunks, Hv, Dk, Dv)))
    for b, h, length in _each(B, T, Hv, lengths):
        S = np.zeros((Dk, Dv)) if init is None else init[b, h]
        err = np.zeros(Dv)
        for c in range(chunks):
            st[0, b, c, h], st[1, b, c, h] = S, _spread(err, Dk)
            at = slice(c * CHUNK, min(length, (c + 1) * CHUNK))
            if at.stop <= at.start:
                continue
            ch = _Chunk(q[b, at, h // share], k[b, at, h // share], v[b, at, h], g[b, at, h], beta[b, at, h], scale)
            s = Num(S)
            u = ch.u(s)
            out = ch.since * scale * ch.q.product(s, more) + ch.P.product(u, more)
            # what the state's error makes of o, by rows: o = N S + ...
            N = scale * ch.since.v * ch.q.v - ch.P.v @ ch.inverse @ (ch.beta.v * ch.since.v * ch.k.v)
            o[0, b, at, h] = out.v
            o[1, b, at, h] = out.e + np.sqrt((N * N).sum(1))[:, None] * err[None, :]
            new = s * ch.whole + (ch.k.T @ (ch.left * u))
            err = np.linalg.norm(ch.map(), 2) * err + np.sqrt((new.e ** 2).sum(0))
            S = new.v
        fin[0, b, h], fin[1, b, h] = S, _spread(err, Dk)
    return Num(*o), Num(*fin), Num(*st)


def backward(q, k, v, g, beta, scale, states, go, gfinal, lengths):
    """Num of the gradients (q, k, v, g, beta, init); `states` as they are handed in."""
    B, T, Hv, Dv = v.shape
    share, Dk = Hv // q.shape[2], q.shape[3]
    chunks = -(-T // CHUNK)
    shapes = (q.shape, q.shape, v.shape, g.shape, g.shape, (B, Hv, Dk, Dv))
    out = [np.zeros((2,) + s) for s in shapes]

    def add(i, at, x):
        out[i][(0,) + at] += x.v
        out[i][(1,) + at] += x.e + (2 * U * np.abs(out[i][(0,) + at]) if i < 2 else 0)

    for b, h, length in _each(B, T, Hv, lengths):
        G = np.zeros((Dk, Dv)) if gfinal is None else gfinal[b, h]
        err = np.zeros(Dv)
        for c in range(chunks - 1, -1, -1):
            at = slice(c * CHUNK, min(length, (c + 1) * CHUNK))
            if at.stop <= at.start:
                continue
            ch = _Chunk(q[b, at, h // share], k[b, at, h // share], v[b, at, h], g[b, at, h], beta[b, at, h], scale)
            S = Num(states[b, c, h], U * np.abs(states[b, c, h]))
            o = Num(go[b, at, h])
            local = Num(G)                       # for the walk: the error so far goes by the map's norm
            gs = Num(G, _spread(err, Dk))        # for this chunk's own gradients
            read, u = ch.read(S), ch.u(S)
            walk = ch.solve(ch.P.T @ o + ch.left * (ch.k @ local), turned=True)
            # the error of dS' reaches dR through a matrix of its own
            N = ch.inverse.T @ (ch.left.v * ch.k.v)
            r = Num(walk.v, walk.e + np.sqrt((N * N).sum(1))[:, None] * err[None, :])
            ru, ou = r @ u.T, o @ u.T
            dP = ou * ch.D * scale
            E = -(ru * ch.beta * ch.strict)
            dq = ch.since * scale * (o @ S.T) + dP @ ch.k
            reads = E @ ch.k - ch.beta * ch.since * (r @ S.T)
            held = ch.left * (u @ gs.T)
            writes = dP.T @ ch.q + E.T @ ch.k + held
            head = (b, at, h // share)
            add(0, head, dq)
            add(1, head, reads + writes)
            add(2, (b, at, h), ch.beta * r)
            add(4, (b, at, h), (r * read).sum(1) - (ru * ch.strict * ch.kk).sum(1))
            dG = (dq * ch.q).sum(1) + ((reads - writes) * ch.k).sum(1)
            last = (S * gs * ch.whole).sum(1).sum(0) + (held * ch.k).sum(1).sum(0)
            dG.v[-1] += last.v
            dG = Num(dG.v, dG.e + np.where(np.arange(len(dG.v)) == len(dG.v) - 1, last.e, 0))
            turn = np.tri(len(dG.v)).T
            add(3, (b, at, h), Num(turn @ dG.v, turn @ dG.e))
            new = local * ch.whole + ch.q.T @ (ch.since * o * scale) - ch.k.T @ (ch.beta * ch.since * walk)
            err = np.linalg.norm(ch.map(), 2) * err + np.sqrt((new.e ** 2).sum(0))
            G = new.v
        out[5][0, b, h], out[5][1, b, h] = G, _spread(err, Dk)
    return [Num(*x) for x in out]


def close(got, want, kind, name):
    """Within the bounds, and as a whole within what roundings of random sign make: errors of a few U
    for each of the some dozens of products that a result goes through, 64 U of the result's size, and
    the result's own rounding."""
    got = np.asarray(got, np.float64)
    assert got.shape == want.v.shape, (name, got.shape, want.v.shape)
    assert np.isfinite(got).all(), name
    d = np.abs(got - want.v)
    bar = want.e * 1.001 + HALF[kind] * (np.abs(want.v) + want.e) + TINY
    assert (d <= bar).all(), (name, float((d - bar).max()), float((d / (bar + 1e-300)).max()), np.argwhere(d > bar)[:5])
    size = np.sqrt((want.v ** 2).mean()) if want.v.size else 0.0
    if size > 0:
        off = np.sqrt((d ** 2).mean()) / size
        assert off <= HALF[kind] + 64 * U, (name, off)
