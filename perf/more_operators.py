"""The gated delta rule and the norms around a block, as cases to be measured: the rule over whole sequences, over one or a few tokens on
its state, and its gradients; the per-head norm of its outputs fused with their gate; the norm after a block fused with the residual's
scaled addition and the norm before the next block; the gradients of both norms.

`run` computes a case in plain torch operations, or, where `own` is set, through the library's entry points.
"""

import math

import torch

own = False

CHUNK = 64            # tokens between two stored states of the delta rule
EPS = 1e-6            # the norms' epsilon
BLOCK = 128           # values that share one 8-bit scale
E4M3_MAX = 448.0
TINY_SCALE = 2.0 ** -126
SCALE = 0.25          # of a block's output as it joins the residual stream
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"

# 65536 tokens are 32 sequences of 2048, the network's training load; its width of 1024 is 16 heads of 64.
LARGEST_ELEMENTS = 65536 * 1024
LARGEST_CHUNK_HEADS = 65536 * 16 // 64  # chunks of 64 tokens times heads, in one case


def listed():
    return [
        # one token for each of 64 sequences that are being generated: a step on the state, in and out
        dict(name="delta step", op="delta", B=64, T=1, Hk=16, Hv=16, Dk=64, Dv=64, dtype="bf16", packed=True, state=True, lengths=False, states=False),
        # five drafted tokens of 16 sequences, two value heads to a key head, wide heads
        dict(name="delta drafted", op="delta", B=16, T=5, Hk=8, Hv=16, Dk=128, Dv=128, dtype="bf16", packed=False, state=True, lengths=False, states=False),
        # the rule of one layer in training: its outputs, and the states that its backward pass starts from
        dict(name="delta layer", op="delta", B=32, T=2048, Hk=16, Hv=16, Dk=64, Dv=64, dtype="bf16", packed=True, state=False, lengths=False, states=True),
        # a padded batch of long prompts being read, shared key heads, wide heads
        dict(name="delta long ragged", op="delta", B=3, T=16411, Hk=4, Hv=8, Dk=128, Dv=128, dtype="bf16", packed=False, state=True, lengths=True, states=False),
        # the gradients of the layer
        dict(name="delta layer backward", op="delta_backward", B=32, T=2048, Hk=16, Hv=16, Dk=64, Dv=64, dtype="bf16", packed=True, lengths=False, final=False),
        # gradients in float32 of a small padded batch: odd head widths, shared key heads, a gradient of the final state
        dict(name="delta odd backward", op="delta_backward", B=2, T=1531, Hk=3, Hv=6, Dk=72, Dv=100, dtype="f32", packed=False, lengths=True, final=True),
        # the rule's outputs of one training batch normed by heads and gated, in 8 bits for the product that follows
        dict(name="gated norm layer", op="gated_norm", rows=65536, H=16, D=64, dtype="bf16", y=False, fp8=True),
        # the same for the tokens of eight sequences that are being generated
        dict(name="gated norm tokens", op="gated_norm", rows=8, H=16, D=64, dtype="bf16", y=False, fp8=True),
        # its gradients, one training batch
        dict(name="gated norm backward", op="gated_norm_backward", rows=65536, H=16, D=64, dtype="bf16"),
        # the end of a block and the start of the next, one training batch: two norms and the residual stream between them
        dict(name="block norm layer", op="block_norm", rows=65536, F=1024, dtype="bf16", y=False, fp8=True),
        # the same for the tokens of eight sequences that are being generated
        dict(name="block norm tokens", op="block_norm", rows=8, F=1024, dtype="bf16", y=False, fp8=True),
        # its gradients, one training batch
        dict(name="block norm backward", op="block_norm_backward", rows=65536, F=1024, dtype="bf16", residual=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "delta_backward", "delta_backward", "gated_norm", "gated_norm_backward", "block_norm", "block_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    elements = LARGEST_ELEMENTS if dtype == "bf16" else LARGEST_ELEMENTS // 2
    if op in ("delta", "delta_backward"):
        Dk, Dv = _log(rng, 16, 128), _log(rng, 16, 128)
        if rng.random() < 0.6:
            Dk, Dv = max(16, Dk // 16 * 16), max(16, Dv // 16 * 16)
        Hk, share = _log(rng, 1, 16), rng.choice([1, 1, 2, 4])
        Hv, B = Hk * share, _log(rng, 1, 64)
        most = LARGEST_CHUNK_HEADS * 64 // (B * Hv) // (4 if Dk > 64 or Dv > 64 else 1) // (1 if dtype == "bf16" else 2)
        T = _log(rng, 1, max(1, min(16411, most)))
        case = dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, packed=rng.random() < 0.5, lengths=rng.random() < 0.4)
        if op == "delta":
            case.update(state=rng.random() < 0.6, states=rng.random() < 0.4)
        else:
            case.update(final=rng.random() < 0.5)
        return case
    if op in ("gated_norm", "gated_norm_backward"):
        D, H = _log(rng, 16, 256), _log(rng, 1, 32)
        if rng.random() < 0.7:
            D = max(16, D // 16 * 16)
        case = dict(op=op, rows=_log(rng, 1, elements // (H * D)), H=H, D=D, dtype=dtype)
    else:
        F = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            F = max(64, F // 64 * 64)
        case = dict(op=op, rows=_log(rng, 1, elements // F), F=F, dtype=dtype)
        if op == "block_norm_backward":
            case["residual"] = rng.random() < 0.7
    if op in ("gated_norm", "block_norm"):
        case["fp8"] = rng.random() < 0.6
        case["y"] = not case["fp8"] or rng.random() < 0.4
    return case


# ------------------------------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _delta_inputs(case, g):
    B, T, Hk, Hv, Dk, Dv, t = (case[k] for k in ("B", "T", "Hk", "Hv", "Dk", "Dv", "dtype"))
    t = TYPES[t]
    if case["packed"]:  # views of one matrix of rows [ q | k | v ]
        rows = torch.empty(B, T, 2 * Hk * Dk + Hv * Dv, device=DEV, dtype=t)
        q, k, v = (w.unflatten(-1, (-1, d)) for w, d in zip(rows.split([Hk * Dk, Hk * Dk, Hv * Dv], -1), (Dk, Dk, Dv)))
    else:
        q, k, v = (torch.empty(B, T, h, d, device=DEV, dtype=t) for h, d in ((Hk, Dk), (Hk, Dk), (Hv, Dv)))
    for w in (q, k):  # what an activation leaves, each head's row scaled to length 1
        w.copy_(torch.nn.functional.normalize(torch.nn.functional.silu(_randn(g, *w.shape)), dim=-1))
    v.copy_(torch.nn.functional.silu(_randn(g, *v.shape, scale=2.0)))
    # log decays as a step width (1e-3 to 1e-1 for each head, moved by the token) times a rate of 1 to 16
    rate = 1 + 15 * torch.rand(Hv, generator=g, device=DEV)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(Hv, generator=g, device=DEV))
    decay = -rate * torch.nn.functional.softplus(_randn(g, B, T, Hv) + torch.log(torch.expm1(step)))
    beta = torch.sigmoid(_randn(g, B, T, Hv, scale=1.5))
    lengths = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32) if case["lengths"] else None
    return dict(q=q, k=k, v=v, g=decay, beta=beta, lengths=lengths)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if op in ("delta", "delta_backward"):
        B, T, Hv, Dk, Dv = (case[k] for k in ("B", "T", "Hv", "Dk", "Dv"))
        s.update(_delta_inputs(case, g))
        start = _randn(g, B, Hv, Dk, Dv, scale=0.3)
        if op == "delta":
            s["initial_state"] = start if case["state"] else None
        else:
            s["chunk_states"] = _plain_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], start, s["lengths"])[2]
            s["grad_o"] = _randn(g, B, T, Hv, Dv, dtype=TYPES[case["dtype"]])
            s["grad_final"] = _randn(g, B, Hv, Dk, Dv) if case["final"] else None
        return s
    R, t = case["rows"], TYPES[case["dtype"]]
    if op in ("gated_norm", "gated_norm_backward"):
        H, D = case["H"], case["D"]
        s["x"] = (_randn(g, R, H * D) * torch.exp(_randn(g, R, 1))).to(t)
        s["gate"] = _randn(g, R, H * D, dtype=t, scale=1.5)
        s["weight"] = 1 + 0.1 * _randn(g, D)
        if op == "gated_norm_backward":
            s["rstd"] = torch.rsqrt(s["x"].float().view(R, H, D).square().mean(2) + EPS)
            s["grad_y"] = _randn(g, R, H * D, dtype=t)
        return s
    F = case["F"]
    s["x"] = (_randn(g, R, F) * torch.exp(_randn(g, R, 1))).to(t)
    s["post_weight"], s["pre_weight"] = 1 + 0.1 * _randn(g, F), 1 + 0.1 * _randn(g, F)
    stream = _randn(g, R, F, dtype=t, scale=2.0)
    if op == "block_norm":
        s["residual"] = stream
    else:
        r = _plain_block_norm(s["x"], stream, s["post_weight"], s["pre_weight"], True, False)
        s["s"], s["post_rstd"], s["pre_rstd"] = r["residual"], r["post_rstd"], r["pre_rstd"]
        s["grad_y"] = _randn(g, R, F, dtype=t)
        s["grad_residual"] = _randn(g, R, F, dtype=t) if case["residual"] else None
    return s


# ------------------------------------------------------------------------------------------------ the plain forms

def _chunked(x, n):
    """(B, T, H, ...) as (B, H, chunks, n, ...), zeros past the end."""
    B, T = x.shape[:2]
    x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, -T % n))
    return x.unflatten(1, (-1, n)).movedim(3, 1)


def _joined(x, T):
    """The other way round."""
    return x.movedim(1, 3).flatten(1, 2)[:, :T]


class _Delta:
    """What both directions form of each chunk, in 32 bits: inside it, a token's u is what it adds to the state along its key."""

    def __init__(self, q, k, v, g, beta, lengths):
        B, T, Hv = g.shape
        n = self.n = min(CHUNK, T)
        share = Hv // k.shape[2]
        if lengths is not None:
            past = torch.arange(T, device=g.device)[None, :] >= lengths[:, None]
            g, beta = (torch.where(past[..., None], 0.0, w) for w in (g, beta))
            q, k, v = (torch.where(past[..., None, None], 0.0, w.float()) for w in (q, k, v))
        self.q, self.k = (_chunked(w.float().repeat_interleave(share, 2), n) for w in (q, k))
        self.v = _chunked(v.float(), n)
        self.beta = _chunked(beta, n)
        sums = _chunked(g, n).double().cumsum(-1)  # in 64 bits: their differences are what counts
        row = torch.arange(n, device=g.device)
        below = row[:, None] >= row[None, :]
        self.strict = row[:, None] > row[None, :]
        self.decay = torch.where(below, (sums[..., :, None] - sums[..., None, :]).clamp_max(0.0).exp(), 0.0).float()
        self.since = sums.exp().float()[..., None]
        self.left = (sums[..., -1:] - sums).exp().float()[..., None]
        self.whole = sums[..., -1].exp().float()[..., None, None]
        self.kk = (self.k @ self.k.mT) * torch.where(self.strict, self.decay, 0.0)
        a = self.beta[..., None] * self.kk
        self.inverse = torch.eye(n, device=g.device).expand_as(a).clone()
        for i in range(1, n):  # of I + a, row by row
            self.inverse[..., i, :i] = -(a[..., i:i + 1, :i] @ self.inverse[..., :i, :i])[..., 0, :]
        self.w = self.inverse @ (self.beta[..., None] * self.since * self.k)
        self.u = self.inverse @ (self.beta[..., None] * self.v)

    def states(self, start):
        """The state before each chunk and after the last."""
        into, s = (self.left * self.k).mT.contiguous(), [start]
        for c in range(self.u.shape[2]):
            u = self.u[:, :, c] - self.w[:, :, c] @ s[-1]
            s.append(self.whole[:, :, c] * s[-1] + into[:, :, c] @ u)
        return torch.stack(s, 2)


def _plain_delta(q, k, v, g, beta, start, lengths):
    B, T, Hv = g.shape
    d = _Delta(q, k, v, g, beta, lengths)
    if start is None:
        start = torch.zeros(B, Hv, k.shape[-1], v.shape[-1], device=g.device)
    s = d.states(start)
    u = d.u - d.w @ s[:, :, :-1]
    o = d.since * (d.q @ s[:, :, :-1]) + (d.q @ d.k.mT * d.decay) @ u
    o = _joined(o * k.shape[-1] ** -0.5, T)
    return o.to(v.dtype), s[:, :, -1].clone(), s[:, :, :-1].transpose(1, 2).contiguous()


def _plain_delta_backward(q, k, v, g, beta, states, lengths, grad_o, grad_final):
    T, share, scale = q.shape[1], v.shape[2] // k.shape[2], k.shape[-1] ** -0.5
    d = _Delta(q, k, v, g, beta, lengths)
    s = states.transpose(1, 2)
    go = grad_o.float() * scale
    if lengths is not None:
        go = torch.where((torch.arange(T, device=g.device)[None, :] >= lengths[:, None])[..., None, None], 0.0, go)
    go = _chunked(go, d.n)
    p = d.q @ d.k.mT * d.decay
    read = d.v - d.since * (d.k @ s)
    u = d.inverse @ (d.beta[..., None] * read)
    # backwards over the chunks: the gradient of the state after each one
    direct, qt = p.mT @ go, (d.since * d.q).mT @ go
    inverse_t, back = d.inverse.mT.contiguous(), (d.beta[..., None] * d.since * d.k).mT.contiguous()
    gs = [torch.zeros_like(s[:, :, 0]) if grad_final is None else grad_final]
    gr = []
    for c in range(s.shape[2] - 1, -1, -1):
        gu = direct[:, :, c] + d.left[:, :, c] * (d.k[:, :, c] @ gs[-1])
        gr.append(inverse_t[:, :, c] @ gu)
        gs.append(d.whole[:, :, c] * gs[-1] + qt[:, :, c] - back[:, :, c] @ gr[-1])
    gr = torch.stack(gr[::-1], 2)
    start = gs.pop()
    gs = torch.stack(gs[::-1], 2)
    gp = (go @ u.mT) * d.decay
    e = -(gr @ u.mT) * d.beta[..., None] * torch.where(d.strict, d.decay, 0.0)
    gq = d.since * (go @ s.mT) + gp @ d.k
    reads = e @ d.k - d.beta[..., None] * d.since * (gr @ s.mT)
    held = d.left * (u @ gs.mT)
    writes = e.mT @ d.k + gp.mT @ d.q + held
    gbeta = (gr * read).sum(-1) - ((gr @ u.mT) * d.kk).sum(-1)
    sums = (gq * d.q).sum(-1) + ((reads - writes) * d.k).sum(-1)
    sums[..., -1] += (d.whole * s * gs).sum((-2, -1)) + (held * d.k).sum((-2, -1))
    gg = sums.double().flip(-1).cumsum(-1).flip(-1).float()
    gq, gk = (_joined(w, T).unflatten(2, (-1, share)).sum(3).to(v.dtype) for w in (gq, reads + writes))
    gv, gg, gbeta = (_joined(w, T) for w in (d.beta[..., None] * gr, gg, gbeta))
    if lengths is not None:
        past = torch.arange(T, device=g.device)[None, :] >= lengths[:, None]
        gg, gbeta = (torch.where(past[..., None], 0.0, w) for w in (gg, gbeta))
        gq, gk, gv = (torch.where(past[..., None, None], 0.0, w) for w in (gq, gk, gv))
    return [gq, gk, gv.to(v.dtype), gg, gbeta, start]


def _plain_quantise(x):
    """e4m3 values and scales of x (R, C) in blocks of 1 x 128."""
    R, C = x.shape
    p = torch.nn.functional.pad(x, (0, -C % BLOCK)).reshape(R, -1, BLOCK)
    scale = (p.abs().amax(2) / E4M3_MAX).clamp_min(TINY_SCALE)
    q = (p / scale[..., None]).reshape(R, -1)[:, :C].to(torch.float8_e4m3fn).contiguous()
    return q, scale.t().contiguous()


def _plain_gated_norm(x, gate, weight, y, fp8):
    D = weight.shape[0]
    v = x.float().unflatten(1, (-1, D))
    rstd = torch.rsqrt(v.square().mean(2) + EPS)
    v = (v * rstd[..., None] * weight).flatten(1) * torch.nn.functional.silu(gate.float())
    out = {"y": v.to(x.dtype) if y else None, "rstd": rstd}
    if fp8:
        out["q"], out["scale"] = _plain_quantise(v)
    return out


def _plain_gated_norm_backward(x, gate, weight, rstd, grad_y):
    D = weight.shape[0]
    n = x.float().unflatten(1, (-1, D)) * rstd[..., None]
    z, gy = (w.float().unflatten(1, (-1, D)) for w in (gate, grad_y))
    sig = torch.sigmoid(z)
    gn = gy * z * sig  # by the normed and weighted values
    gw = (gn.double() * n.double()).sum((0, 1)).float()
    gz = gy * n * weight * sig * (1 + z * (1 - sig))
    gn = gn * weight
    gx = rstd[..., None] * (gn - n * (gn * n).mean(2, keepdim=True))
    return {"x": gx.flatten(1).to(x.dtype), "gate": gz.flatten(1).to(x.dtype), "weight": gw}


def _plain_block_norm(x, residual, post_weight, pre_weight, y, fp8):
    x = x.float()
    post = torch.rsqrt(x.square().mean(1) + EPS)
    s = residual.float() + SCALE * (x * post[:, None] * post_weight)
    pre = torch.rsqrt(s.square().mean(1) + EPS)
    v = s * pre[:, None] * pre_weight
    out = {"y": v.to(residual.dtype) if y else None, "residual": s.to(residual.dtype), "post_rstd": post, "pre_rstd": pre}
    if fp8:
        out["q"], out["scale"] = _plain_quantise(v)
    return out


def _plain_block_norm_backward(x, s, post_weight, pre_weight, post_rstd, pre_rstd, grad_y, grad_residual):
    m, n, gy = s.float() * pre_rstd[:, None], x.float() * post_rstd[:, None], grad_y.float()
    gpre = (gy.double() * m.double()).sum(0).float()
    gm = gy * pre_weight
    gs = pre_rstd[:, None] * (gm - m * (gm * m).mean(1, keepdim=True))
    if grad_residual is not None:
        gs = gs + grad_residual.float()
    ga = SCALE * gs
    gpost = (ga.double() * n.double()).sum(0).float()
    gn = ga * post_weight
    gx = post_rstd[:, None] * (gn - n * (gn * n).mean(1, keepdim=True))
    return {"x": gx.to(x.dtype), "residual": gs.to(x.dtype), "post_weight": gpost, "pre_weight": gpre}


def run(state):
    if own:
        return _run_own(state)
    s, c = state, state["case"]
    if s["op"] == "delta":
        o, final, states = _plain_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["initial_state"], s["lengths"])
        return {"o": o, "final": final, "states": states if c["states"] else None}
    if s["op"] == "delta_backward":
        return _plain_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["chunk_states"], s["lengths"], s["grad_o"], s["grad_final"])
    if s["op"] == "gated_norm":
        return _plain_gated_norm(s["x"], s["gate"], s["weight"], c["y"], c["fp8"])
    if s["op"] == "gated_norm_backward":
        return _plain_gated_norm_backward(s["x"], s["gate"], s["weight"], s["rstd"], s["grad_y"])
    if s["op"] == "block_norm":
        return _plain_block_norm(s["x"], s["residual"], s["post_weight"], s["pre_weight"], c["y"], c["fp8"])
    return _plain_block_norm_backward(s["x"], s["s"], s["post_weight"], s["pre_weight"], s["post_rstd"], s["pre_rstd"], s["grad_y"], s["grad_residual"])


def _run_own(s):
    import complex_chunkwise_ssd_amd as ssd

    c = s["case"]
    if s["op"] == "delta":
        r = ssd.gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], initial_state=s["initial_state"], lengths=s["lengths"],
                            want_chunk_states=c["states"])
        return {"o": r.o, "final": r.final_state, "states": r.chunk_states}
    if s["op"] == "delta_backward":
        r = ssd.gated_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["chunk_states"], s["grad_o"], grad_final_state=s["grad_final"],
                                     lengths=s["lengths"])
        return [r.q, r.k, r.v, r.g, r.beta, r.initial_state]
    if s["op"] == "gated_norm":
        r = ssd.gated_norm(s["x"], s["gate"], s["weight"], eps=EPS, want_y=c["y"], fp8=c["fp8"], want_rstd=True)
        out = {"y": r.y, "rstd": r.rstd}
    elif s["op"] == "gated_norm_backward":
        gx, gz, gw = ssd.gated_norm_backward(s["x"], s["gate"], s["weight"], s["rstd"], s["grad_y"])
        return {"x": gx, "gate": gz, "weight": gw}
    elif s["op"] == "block_norm":
        r = ssd.block_norm(s["x"], s["residual"], s["post_weight"], s["pre_weight"], residual_scale=SCALE, eps=EPS, want_y=c["y"], fp8=c["fp8"],
                           want_rstd=True)
        out = {"y": r.y, "residual": r.residual, "post_rstd": r.post_rstd, "pre_rstd": r.pre_rstd}
    else:
        gx, gs, gpost, gpre = ssd.block_norm_backward(s["x"], s["s"], s["post_weight"], s["pre_weight"], s["post_rstd"], s["pre_rstd"], s["grad_y"],
                                                      grad_residual=s["grad_residual"], residual_scale=SCALE)
        return {"x": gx, "residual": gs, "post_weight": gpost, "pre_weight": gpre}
    if c["fp8"]:
        out["q"], out["scale"] = r.q, r.scale
    return out


# ------------------------------------------------------------------------------------------ the definitions in 64 bits

class _Tokens:
    """The delta rule one token after the other, in 64 bits: (B, H, D) of each token, the state (B, H, Dk, Dv)."""

    def __init__(self, s):
        case = s["case"]
        share = case["Hv"] // case["Hk"]
        self.T, self.scale = case["T"], case["Dk"] ** -0.5
        self.valid = None if s["lengths"] is None else torch.arange(self.T, device=DEV)[:, None] < s["lengths"][None, :]  # (T, B)
        heads = lambda w: w.transpose(0, 1).double().repeat_interleave(share, 2)  # noqa: E731
        self.q, self.k, self.v = heads(s["q"]), heads(s["k"]), s["v"].transpose(0, 1).double()
        self.a, self.b = torch.exp(s["g"].transpose(0, 1).double()), s["beta"].transpose(0, 1).double()
        if self.valid is not None:
            dead = ~self.valid
            self.a[dead], self.b[dead] = 1.0, 0.0
            self.q[dead], self.k[dead], self.v[dead] = 0.0, 0.0, 0.0

    def step(self, t, S):
        """(decayed state, what the key read from it, what it adds, new state)"""
        D = S * self.a[t][..., None, None]
        p = torch.einsum("bhkv,bhk->bhv", D, self.k[t])
        u = self.b[t][..., None] * (self.v[t] - p)
        return D, p, u, torch.addcmul(D, self.k[t][..., :, None], u[..., None, :])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "delta":
        d = _Tokens(s)
        S = torch.zeros(case["B"], case["Hv"], case["Dk"], case["Dv"], dtype=torch.float64, device=DEV) if s["initial_state"] is None else s["initial_state"].double()
        o, states = [], []
        for t in range(case["T"]):
            if t % CHUNK == 0 and case["states"]:
                states.append(S)
            S = d.step(t, S)[3]
            o.append(torch.einsum("bhkv,bhk->bhv", S, d.q[t]) * d.scale)
        return {"o": torch.stack(o, 1), "final": S, "states": torch.stack(states, 1) if states else None}
    if op == "delta_backward":
        d, T, share = _Tokens(s), case["T"], case["Hv"] // case["Hk"]
        go = s["grad_o"].transpose(0, 1).double() * d.scale
        if d.valid is not None:
            go[~d.valid] = 0.0
        gs = torch.zeros_like(s["chunk_states"][:, 0], dtype=torch.float64) if s["grad_final"] is None else s["grad_final"].double()
        out = [torch.empty_like(w) for w in (d.q, d.k, d.v, d.a, d.b)]
        S = s["chunk_states"][:, 0].double()
        starts = []
        for t in range(T):
            if t % CHUNK == 0:
                starts.append(S)
            S = d.step(t, S)[3]
        for c in range(len(starts) - 1, -1, -1):
            seen, S = [], starts[c]
            for t in range(c * CHUNK, min(T, (c + 1) * CHUNK)):
                seen.append(d.step(t, S))
                S = seen[-1][3]
            for t in range(min(T, (c + 1) * CHUNK) - 1, c * CHUNK - 1, -1):
                D, p, u, S = seen.pop()
                gs = torch.addcmul(gs, d.q[t][..., :, None], go[t][..., None, :])
                gu = torch.einsum("bhkv,bhk->bhv", gs, d.k[t])
                w = -d.b[t][..., None] * gu
                out[0][t] = torch.einsum("bhkv,bhv->bhk", S, go[t])
                out[1][t] = torch.einsum("bhkv,bhv->bhk", gs, u) + torch.einsum("bhkv,bhv->bhk", D, w)
                out[2][t] = -w
                out[4][t] = (gu * (d.v[t] - p)).sum(-1)
                gs = torch.addcmul(gs, d.k[t][..., :, None], w[..., None, :])
                out[3][t] = (gs * D).sum((-2, -1))
                gs = gs * d.a[t][..., None, None]
        if d.valid is not None:
            for w in out:
                w[~d.valid] = 0.0
        out = [w.transpose(0, 1) for w in out]
        out[:2] = [w.unflatten(2, (-1, share)).sum(3) for w in out[:2]]
        return out + [gs]
    if op == "gated_norm":
        x, z, w = s["x"].double(), s["gate"].double(), s["weight"].double()
        x = x.view(case["rows"], case["H"], case["D"])
        rms = torch.sqrt((x * x).sum(2) / case["D"] + EPS)
        y = (x / rms[..., None] * w).reshape(case["rows"], -1) * z / (1 + torch.exp(-z))
        out = {"y": y if case["y"] else None, "rstd": 1 / rms}
    elif op == "gated_norm_backward":
        R, H, D = case["rows"], case["H"], case["D"]
        x, z, gy = (s[k].double().view(R, H, D) for k in ("x", "gate", "grad_y"))
        w, r = s["weight"].double(), s["rstd"].double()[..., None]
        act = z / (1 + torch.exp(-z))
        slope = (1 + torch.exp(-z) * (1 + z)) / (1 + torch.exp(-z)) ** 2
        by_n = gy * act * w
        gx = r * by_n - x * r ** 3 * (by_n * x).sum(2, keepdim=True) / D
        return {"x": gx.view(R, H * D), "gate": (gy * x * r * w * slope).view(R, H * D), "weight": (gy * act * x * r).sum((0, 1))}
    elif op == "block_norm":
        x, res = s["x"].double(), s["residual"].double()
        post = torch.sqrt((x * x).sum(1, keepdim=True) / case["F"] + EPS)
        stream = res + SCALE * s["post_weight"].double() * x / post
        pre = torch.sqrt((stream * stream).sum(1, keepdim=True) / case["F"] + EPS)
        y = stream / pre * s["pre_weight"].double()
        out = {"y": y if case["y"] else None, "residual": stream, "post_rstd": 1 / post[:, 0], "pre_rstd": 1 / pre[:, 0]}
    else:
        F = case["F"]
        x, stream, gy = s["x"].double(), s["s"].double(), s["grad_y"].double()
        a, b = s["post_rstd"].double()[:, None], s["pre_rstd"].double()[:, None]
        by_m = gy * s["pre_weight"].double()
        gs = b * by_m - stream * b ** 3 * (by_m * stream).sum(1, keepdim=True) / F
        if s["grad_residual"] is not None:
            gs = gs + s["grad_residual"].double()
        by_n = SCALE * gs * s["post_weight"].double()
        gx = a * by_n - x * a ** 3 * (by_n * x).sum(1, keepdim=True) / F
        return {"x": gx, "residual": gs, "post_weight": (SCALE * gs * x * a).sum(0), "pre_weight": (gy * stream * b).sum(0)}
    if case["fp8"]:
        R, C = y.shape
        p = torch.zeros(R, -(-C // BLOCK) * BLOCK, dtype=torch.float64, device=DEV)
        p[:, :C] = y
        scale = torch.clamp(p.abs().view(R, -1, BLOCK).amax(2) / E4M3_MAX, min=TINY_SCALE)
        v = p / scale.repeat_interleave(BLOCK, 1)
        step = torch.ldexp(torch.ones_like(v), torch.clamp(torch.frexp(v)[1] - 1, min=-6) - 3)
        out["q"], out["scale"] = (torch.round(v / step) * step)[:, :C], scale.t()
    return out


# ------------------------------------------------------------------------------------------ what a case has to move and do

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("delta", "delta_backward"):
        B, T, Hk, Hv, Dk, Dv = (case[k] for k in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
        keys, values, gates, state = e * B * T * Hk * Dk, e * B * T * Hv * Dv, 4 * B * T * Hv, 4 * B * Hv * Dk * Dv
        stored = state * -(-T // CHUNK)
        if op == "delta":
            return {"bytes": 2 * keys + 2 * values + 2 * gates + state * (1 + case["state"]) + (stored if case["states"] else 0), "flops": 7 * B * T * Hv * Dk * Dv}
        return {"bytes": 4 * keys + 3 * values + 4 * gates + stored + state * (1 + case["final"]), "flops": 21 * B * T * Hv * Dk * Dv}
    F = case["F"] if "F" in case else case["H"] * case["D"]
    n = case["rows"] * F
    if op in ("gated_norm", "block_norm"):
        moved = e * (2 + case["y"] + (op == "block_norm")) * n + (n + 4 * case["rows"] * -(-F // BLOCK) if case["fp8"] else 0)
        return {"bytes": moved + 4 * case["rows"] * (case["H"] if "H" in case else 2) + (4 * case["D"] if "D" in case else 8 * F), "flops": 12 * n}
    if op == "gated_norm_backward":
        return {"bytes": 5 * e * n + 4 * case["rows"] * case["H"] + 8 * case["D"], "flops": 24 * n}
    return {"bytes": (5 + case["residual"]) * e * n + 8 * case["rows"] + 16 * F, "flops": 20 * n}
