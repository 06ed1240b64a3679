"""The operators around the scan, as cases to be measured: the gated linear recurrence, the RMS norm with the residual's
addition and 8-bit output, the 8-bit quantisation by blocks of 128 and the matrix product of such operands.

`run` computes a case in plain torch operations, or, where `own` is set, through the library's entry points.
"""

import math

import torch

own = False

CHUNK = 64            # tokens between two stored states of the gated scan
DECAY = 8.0           # the gated scan's decay scale
EPS = 1e-6            # the norm's epsilon
BLOCK = 128           # values that share one 8-bit scale
E4M3_MAX = 448.0
TINY_SCALE = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"

# 65536 tokens are 32 sequences of 2048, the network's training load; 1024 is its width, 5136 = 16 (64 + 4 * 64 + 1)
# the width of its in_proj rows.
LARGEST_FLOPS = 2 * 65536 * 5136 * 1024
LARGEST_ELEMENTS = 65536 * 1024


def listed():
    return [
        # one token for each of 64 sequences that are being generated: the recurrence's step with the state in and out
        dict(name="gated step", op="gated_scan", B=64, T=1, C=1024, dtype="bf16", packed=False, state=True, lengths=False, states=False),
        # the recurrence of one layer in training: its outputs, and the states that its backward pass starts from
        dict(name="gated layer", op="gated_scan", B=32, T=2048, C=1024, dtype="bf16", packed=False, state=False, lengths=False, states=True),
        # a padded batch of long documents being read, one row of odd length and width, in float32
        dict(name="gated long ragged", op="gated_scan", B=3, T=16411, C=1000, dtype="f32", packed=False, state=True, lengths=True, states=False),
        # the gradients of the layer
        dict(name="gated layer backward", op="gated_scan_backward", B=32, T=2048, C=1024, dtype="bf16", packed=False, lengths=False, final=False),
        # the norm in front of in_proj, one training batch: residual stream updated, rows in 8 bits for the product
        dict(name="norm layer", op="rms_norm", rows=65536, F=1024, dtype="bf16", residual=True, y=False, fp8=True),
        # the same for the tokens of eight sequences that are being generated
        dict(name="norm tokens", op="rms_norm", rows=8, F=1024, dtype="bf16", residual=True, y=False, fp8=True),
        # the gradients of the norm, one training batch
        dict(name="norm layer backward", op="rms_norm_backward", rows=65536, F=1024, dtype="bf16", residual=True),
        # the layer's activations turned for the weight gradient: each channel's tokens in blocks of 128
        dict(name="quantise turned", op="fp8_quantise", rows=65536, cols=1024, dtype="bf16", block_rows=1, transpose=True),
        # the in_proj weight, turned for the input gradient, in blocks of 128 x 128
        dict(name="quantise weight", op="fp8_quantise", rows=5136, cols=1024, dtype="f32", block_rows=128, transpose=True),
        # in_proj of one training batch: its rows in bfloat16, as the scan reads them
        dict(name="in_proj layer", op="fp8_matmul", M=65536, N=5136, K=1024, block_rows=128, out="bf16"),
        # in_proj of the tokens of eight sequences that are being generated
        dict(name="in_proj tokens", op="fp8_matmul", M=8, N=5136, K=1024, block_rows=128, out="bf16"),
        # the weight gradient of in_proj: a sum over every token, scales along the tokens on both sides
        dict(name="in_proj weight gradient", op="fp8_matmul", M=5136, N=1024, K=65536, block_rows=1, out="f32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gated_scan", "gated_scan_backward", "rms_norm", "rms_norm_backward", "fp8_quantise", "fp8_matmul", "fp8_matmul"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    elements = LARGEST_ELEMENTS if dtype == "bf16" else LARGEST_ELEMENTS // 2
    if op in ("gated_scan", "gated_scan_backward"):
        B, C = _log(rng, 1, 64), _log(rng, 16, 4096)
        if rng.random() < 0.6:
            C = max(16, C // 16 * 16)
        T = _log(rng, 1, max(1, min(32768, elements // (B * C))))
        case = dict(op=op, B=B, T=T, C=C, dtype=dtype, packed=rng.random() < 0.5, lengths=rng.random() < 0.4)
        if op == "gated_scan":
            case.update(state=rng.random() < 0.6, states=rng.random() < 0.4)
        else:
            case.update(final=rng.random() < 0.5)
        return case
    if op in ("rms_norm", "rms_norm_backward"):
        F = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            F = max(64, F // 64 * 64)
        case = dict(op=op, rows=_log(rng, 1, elements // F), F=F, dtype=dtype, residual=rng.random() < 0.7)
        if op == "rms_norm":
            case["fp8"] = rng.random() < 0.6
            case["y"] = not case["fp8"] or rng.random() < 0.4
        return case
    if op == "fp8_quantise":
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = max(64, cols // 64 * 64)
        return dict(op=op, rows=_log(rng, 1, elements // cols), cols=cols, dtype=dtype, block_rows=rng.choice([1, 128]), transpose=rng.random() < 0.5)
    N, K = _log(rng, 64, 16384), _log(rng, 64, 16384)
    if rng.random() < 0.7:
        N, K = max(64, N // 16 * 16), max(64, K // 16 * 16)
    M = _log(rng, 1, max(1, min(65536, LARGEST_FLOPS // (2 * N * K), (1 << 28) // N)))
    return dict(op="fp8_matmul", M=M, N=N, K=K, block_rows=rng.choice([128, 128, 1]), out=rng.choice(["bf16", "bf16", "f32"]))


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _gated_inputs(case, g):
    B, T, C, t = case["B"], case["T"], case["C"], TYPES[case["dtype"]]
    if case["packed"]:  # views of projected rows [ x | input gate | decay gate ]
        rows = _randn(g, B, T, 3 * C, dtype=t)
        x, gi, gr = rows[..., :C], rows[..., C:2 * C], rows[..., 2 * C:]
    else:
        x, gi, gr = (_randn(g, B, T, C, dtype=t) for _ in range(3))
    full = torch.rand(C, generator=g, device=DEV, dtype=torch.float64) * 0.099 + 0.9  # the decay at an open gate, 0.9 to 0.999
    lam = torch.log(torch.expm1(-torch.log(full) / DECAY)).float()
    lengths = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32) if case["lengths"] else None
    return dict(x=x, input_gate=gi, decay_gate=gr, lam=lam, lengths=lengths)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "gated_scan":
        s.update(_gated_inputs(case, g))
        s["initial_state"] = _randn(g, case["B"], case["C"]) if case["state"] else None
    elif op == "gated_scan_backward":
        s.update(_gated_inputs(case, g))
        init = _randn(g, case["B"], case["C"])
        s["chunk_states"] = _plain_gated(s["x"], s["input_gate"], s["decay_gate"], s["lam"], init, s["lengths"])[2]
        s["grad_h"] = _randn(g, case["B"], case["T"], case["C"], dtype=TYPES[case["dtype"]])
        s["grad_final"] = _randn(g, case["B"], case["C"]) if case["final"] else None
    elif op in ("rms_norm", "rms_norm_backward"):
        R, F, t = case["rows"], case["F"], TYPES[case["dtype"]]
        s["x"] = _randn(g, R, F, dtype=t)
        s["weight"] = 1 + 0.1 * _randn(g, F)
        s["residual"] = _randn(g, R, F, dtype=t, scale=2.0) if case["residual"] else None
        if op == "rms_norm_backward":  # x is the sum that the norm was taken of; residual the gradient of the residual stream
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["grad_y"] = _randn(g, R, F, dtype=t)
    elif op == "fp8_quantise":
        s["x"] = _randn(g, case["rows"], case["cols"], dtype=TYPES[case["dtype"]]) * torch.exp(_randn(g, case["rows"], 1)).to(TYPES[case["dtype"]])
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["a_scale"] = _plain_quantise(_randn(g, M, K, dtype=torch.bfloat16), 1, False)
        s["b"], s["b_scale"] = _plain_quantise(_randn(g, N, K, scale=K ** -0.5), case["block_rows"], False)
    return s


# ------------------------------------------------------------------------------------------------ the plain forms

def _plain_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1, by doubling the span of each step."""
    k = 1
    while k < a.shape[1]:
        u = torch.cat([u[:, :k], u[:, k:] + a[:, k:] * u[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return u


def _valid(lengths, T):
    return None if lengths is None else (torch.arange(T, device=lengths.device)[None, :] < lengths[:, None])[..., None]


def _plain_gates(x, gi, gr, lam, valid):
    i, r = torch.sigmoid(gi.float()), torch.sigmoid(gr.float())
    l = -DECAY * torch.nn.functional.softplus(lam) * r
    a, m = torch.exp(l), torch.sqrt(-torch.expm1(2 * l))
    u = m * i * x.float()
    if valid is not None:
        a, u = torch.where(valid, a, 1.0), torch.where(valid, u, 0.0)
    return i, r, l, a, m, u


def _plain_gated(x, gi, gr, lam, init, lengths):
    B, T, C = x.shape
    valid = _valid(lengths, T)
    _, _, _, a, _, u = _plain_gates(x, gi, gr, lam, valid)
    start = torch.zeros(B, C, device=x.device) if init is None else init
    u = torch.cat([(a[:, 0] * start + u[:, 0])[:, None], u[:, 1:]], 1)
    s = _plain_scan(a, u)
    states = torch.cat([start[:, None], s[:, CHUNK - 1:T - 1:CHUNK]], 1)
    h = s if valid is None else torch.where(valid, s, 0.0)
    return h.to(x.dtype), s[:, -1].clone(), states


def _plain_gated_backward(x, gi, gr, lam, states, lengths, grad_h, grad_final):
    B, T, C = x.shape
    valid = _valid(lengths, T)
    i, r, l, a, m, u = _plain_gates(x, gi, gr, lam, valid)
    start = states[:, 0]
    h = _plain_scan(a, torch.cat([(a[:, 0] * start + u[:, 0])[:, None], u[:, 1:]], 1))
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    g = grad_h.float() if valid is None else torch.where(valid, grad_h.float(), 0.0)
    if grad_final is not None:
        g = torch.cat([g[:, :-1], (g[:, -1] + grad_final)[:, None]], 1)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _plain_scan(after.flip(1), g.flip(1)).flip(1)
    grad_init = a[:, 0] * g[:, 0]
    xf = x.float()
    e = g * before * a * l - g * i * xf * a * a * (l / m)
    out = [g * m * i, g * m * xf * i * (1 - i), e * (1 - r)]
    if valid is not None:
        e = torch.where(valid, e, 0.0)
        out = [torch.where(valid, v, 0.0) for v in out]
    lam64 = lam.double()
    grad_lam = (torch.sigmoid(lam64) / torch.nn.functional.softplus(lam64) * e.double().sum((0, 1))).float()
    return [v.to(x.dtype) for v in out] + [grad_lam, grad_init]


def _plain_quantise(x, block_rows, transpose):
    """e4m3 values and scales of x (R, C) in blocks of block_rows x 128 (turned first, where asked)."""
    x = x.float()
    x = x.t() if transpose else x
    R, C = x.shape
    rb = -(-R // block_rows)
    p = torch.nn.functional.pad(x, (0, _blocks(C) * BLOCK - C, 0, rb * block_rows - R)).reshape(rb, block_rows, _blocks(C), BLOCK)
    scale = (p.abs().amax((1, 3)) / E4M3_MAX).clamp_min(TINY_SCALE)
    q = (p / scale[:, None, :, None]).reshape(rb * block_rows, -1)[:R, :C].to(torch.float8_e4m3fn).contiguous()
    return q, scale.t().contiguous() if block_rows == 1 else scale


def _dequantised(q, scale, block_rows, real):
    """The values of q (R, C) with its scales, in the type `real`."""
    scale = scale.to(real)
    full = scale.t() if block_rows == 1 else scale.repeat_interleave(BLOCK, 0)[:q.shape[0]]
    return q.to(real) * full.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _plain_norm(x, weight, residual, y, fp8):
    s = x.float() if residual is None else x.float() + residual.float()
    v = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * weight
    out = {"y": v.to(x.dtype) if y else None, "residual": None if residual is None else s.to(x.dtype)}
    if fp8:
        out["q"], out["scale"] = _plain_quantise(v, 1, False)
    return out


def _plain_norm_backward(s, weight, rstd, grad_y, grad_residual):
    s, gy, rstd = s.float(), grad_y.float(), rstd[:, None]
    gw = (gy.double() * s.double() * rstd.double()).sum(0).float()
    g = rstd * (gy * weight - s * rstd * rstd * (gy * weight * s).mean(1, keepdim=True))
    if grad_residual is not None:
        g = g + grad_residual.float()
    return {"x": g.to(grad_y.dtype), "weight": gw}


def run(state):
    if own:
        return _run_own(state)
    s, c = state, state["case"]
    if s["op"] == "gated_scan":
        h, final, states = _plain_gated(s["x"], s["input_gate"], s["decay_gate"], s["lam"], s["initial_state"], s["lengths"])
        return {"h": h, "final": final, "states": states if c["states"] else None}
    if s["op"] == "gated_scan_backward":
        return _plain_gated_backward(s["x"], s["input_gate"], s["decay_gate"], s["lam"], s["chunk_states"], s["lengths"], s["grad_h"], s["grad_final"])
    if s["op"] == "rms_norm":
        return _plain_norm(s["x"], s["weight"], s["residual"], c["y"], c["fp8"])
    if s["op"] == "rms_norm_backward":
        return _plain_norm_backward(s["x"], s["weight"], s["rstd"], s["grad_y"], s["residual"])
    if s["op"] == "fp8_quantise":
        q, scale = _plain_quantise(s["x"], c["block_rows"], c["transpose"])
        return {"q": q, "scale": scale}
    a = _dequantised(s["a"], s["a_scale"], 1, torch.float32)
    b = _dequantised(s["b"], s["b_scale"], c["block_rows"], torch.float32)
    return (a @ b.t()).to(TYPES[c["out"]])


def _run_own(s):
    import complex_chunkwise_ssd_amd as ssd

    c = s["case"]
    if s["op"] == "gated_scan":
        r = ssd.gated_scan(s["x"], s["input_gate"], s["decay_gate"], s["lam"], decay_scale=DECAY, initial_state=s["initial_state"],
                           lengths=s["lengths"], want_chunk_states=c["states"])
        return {"h": r.h, "final": r.final_state, "states": r.chunk_states}
    if s["op"] == "gated_scan_backward":
        r = ssd.gated_scan_backward(s["x"], s["input_gate"], s["decay_gate"], s["lam"], s["chunk_states"], s["grad_h"],
                                    grad_final_state=s["grad_final"], decay_scale=DECAY, lengths=s["lengths"])
        return [r.x, r.input_gate, r.decay_gate, r.lam, r.initial_state]
    if s["op"] == "rms_norm":
        r = ssd.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, want_y=c["y"], fp8=c["fp8"])
        out = {"y": r.y, "residual": r.residual}
        if c["fp8"]:
            out["q"], out["scale"] = r.q, r.scale
        return out
    if s["op"] == "rms_norm_backward":
        grad_x, grad_weight = ssd.rms_norm_backward(s["x"], s["weight"], s["rstd"], s["grad_y"], grad_residual=s["residual"])
        return {"x": grad_x, "weight": grad_weight}
    if s["op"] == "fp8_quantise":
        q, scale = ssd.fp8_quantise(s["x"], block_rows=c["block_rows"], transpose=c["transpose"])
        return {"q": q, "scale": scale}
    return ssd.fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], block_rows=c["block_rows"], out_dtype=TYPES[c["out"]])


# ------------------------------------------------------------------------------------------ the definitions in 64 bits

def _exact_gates(s):
    sp = torch.logaddexp(s["lam"].double(), torch.zeros((), dtype=torch.float64, device=DEV))
    i = 1 / (1 + torch.exp(-s["input_gate"].double()))
    r = 1 / (1 + torch.exp(-s["decay_gate"].double()))
    l = -DECAY * sp * r
    return sp, i, r, l


def _exact_states(s, start, sp, i, r, l):
    """The state before each token and after the last, in 64 bits, one token after the other."""
    x = s["x"].double()
    B, T, C = x.shape
    a, u = torch.exp(l), torch.sqrt(-torch.expm1(2 * l)) * i * x
    if s["lengths"] is not None:
        dead = torch.arange(T, device=DEV)[None, :] >= s["lengths"][:, None]
        a[dead], u[dead] = 1.0, 0.0
    before = torch.empty(B, T + 1, C, dtype=torch.float64, device=DEV)
    before[:, 0] = start
    for t in range(T):
        torch.addcmul(u[:, t], a[:, t], before[:, t], out=before[:, t + 1])
    return a, before


def _exact_e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantise(v, block_rows):
    """v (R, C) in float64 to e4m3 values (in float64) and scales."""
    R, C = v.shape
    rb, cb = -(-R // block_rows), _blocks(C)
    p = torch.zeros(rb * block_rows, cb * BLOCK, dtype=torch.float64, device=DEV)
    p[:R, :C] = v
    top = p.abs().view(rb, block_rows, cb, BLOCK).amax(dim=(1, 3))
    scale = torch.clamp(top / E4M3_MAX, min=TINY_SCALE)
    q = _exact_e4m3(p / scale.repeat_interleave(block_rows, 0).repeat_interleave(BLOCK, 1))[:R, :C]
    return q, scale.t() if block_rows == 1 else scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated_scan":
        gates = _exact_gates(s)
        start = 0.0 if s["initial_state"] is None else s["initial_state"].double()
        _, before = _exact_states(s, start, *gates)
        h = before[:, 1:].clone()
        if s["lengths"] is not None:
            h[torch.arange(case["T"], device=DEV)[None, :] >= s["lengths"][:, None]] = 0.0
        return {"h": h, "final": before[:, -1], "states": before[:, :-1:CHUNK] if case["states"] else None}
    if op == "gated_scan_backward":
        sp, i, r, l = _exact_gates(s)
        a, before = _exact_states(s, s["chunk_states"][:, 0].double(), sp, i, r, l)
        x, gh = s["x"].double(), s["grad_h"].double()
        dead = None
        if s["lengths"] is not None:
            dead = torch.arange(case["T"], device=DEV)[None, :] >= s["lengths"][:, None]
            gh[dead] = 0.0
        g = torch.empty_like(gh)
        carry = torch.zeros(case["B"], case["C"], dtype=torch.float64, device=DEV) if s["grad_final"] is None else s["grad_final"].double()
        for t in range(case["T"] - 1, -1, -1):
            torch.add(gh[:, t], carry, out=g[:, t])
            carry = a[:, t] * g[:, t]
        m = torch.sqrt(-torch.expm1(2 * l))
        by_l = g * (before[:, :-1] * a - i * x * a * a / m)  # the loss's derivative by l
        out = [g * m * i, g * m * x * i * (1 - i), by_l * l * (1 - r)]
        by_lam = by_l * (-DECAY * r) / (1 + torch.exp(-s["lam"].double()))
        if dead is not None:
            by_lam[dead] = 0.0
            for v in out:
                v[dead] = 0.0
        return out + [by_lam.sum(dim=(0, 1)), carry]
    if op == "rms_norm":
        x, w = s["x"].double(), s["weight"].double()
        if s["residual"] is not None:
            x = x + s["residual"].double()
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / case["F"] + EPS) * w
        out = {"y": y if case["y"] else None, "residual": x if case["residual"] else None}
        if case["fp8"]:
            out["q"], out["scale"] = _exact_quantise(y, 1)
        return out
    if op == "rms_norm_backward":
        x, w, gy, rstd = s["x"].double(), s["weight"].double(), s["grad_y"].double(), s["rstd"].double()[:, None]
        n = x * rstd
        gn = gy * w
        gx = rstd * (gn - n * (gn * n).sum(1, keepdim=True) / case["F"])
        if s["residual"] is not None:
            gx = gx + s["residual"].double()
        return {"x": gx, "weight": (gy * n).sum(0)}
    if op == "fp8_quantise":
        v = s["x"].double()
        q, scale = _exact_quantise(v.t() if case["transpose"] else v, case["block_rows"])
        return {"q": q, "scale": scale}
    M, N, K = case["M"], case["N"], case["K"]
    out = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    wide = 64 * BLOCK
    for k in range(0, K, wide):
        kb = slice(k // BLOCK, (k + wide) // BLOCK)
        sa = s["a_scale"].double()[kb].repeat_interleave(BLOCK, 0).t()
        sb = s["b_scale"].double()
        sb = sb[kb].repeat_interleave(BLOCK, 0).t() if case["block_rows"] == 1 else sb[:, kb].repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:N]
        a, b = s["a"][:, k:k + wide].double(), s["b"][:, k:k + wide].double()
        out += (a * sa[:, :a.shape[1]]) @ (b * sb[:, :b.shape[1]]).t()
    return out


# ------------------------------------------------------------------------------------------ what a case has to move and do

def work(case):
    op, e = case["op"], 2 if case.get("dtype") == "bf16" else 4
    if op in ("gated_scan", "gated_scan_backward"):
        n, bc = case["B"] * case["T"] * case["C"], case["B"] * case["C"]
        stored = 4 * bc * -(-case["T"] // CHUNK)
        if op == "gated_scan":
            return {"bytes": 4 * e * n + 4 * bc * (1 + case["state"]) + (stored if case["states"] else 0), "flops": 30 * n}
        return {"bytes": 7 * e * n + stored + 4 * bc * (1 + case["final"]), "flops": 60 * n}
    if op == "rms_norm":
        n = case["rows"] * case["F"]
        moved = e * (1 + 2 * case["residual"] + case["y"]) * n
        if case["fp8"]:
            moved += n + 4 * case["rows"] * _blocks(case["F"])
        return {"bytes": moved + 4 * case["F"], "flops": 6 * n}
    if op == "rms_norm_backward":
        n = case["rows"] * case["F"]
        return {"bytes": e * (3 + case["residual"]) * n + 8 * case["F"] + 4 * case["rows"], "flops": 12 * n}
    if op == "fp8_quantise":
        n = case["rows"] * case["cols"]
        R, C = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        return {"bytes": (e + 1) * n + 4 * -(-R // case["block_rows"]) * _blocks(C), "flops": 3 * n}
    M, N, K = case["M"], case["N"], case["K"]
    kb = _blocks(K)
    scales = 4 * kb * (M + (N if case["block_rows"] == 1 else _blocks(N)))
    return {"bytes": (M + N) * K + scales + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
