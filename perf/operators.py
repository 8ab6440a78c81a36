"""The workloads of the channelwise recurrence, the layer norm and the 8-bit
activation checkpoints: their inputs, one pass through each operator in plain
torch and through the library, their least traffic and their 64-bit values.

Widths follow the framework's layer workload (16 heads of 128 channels: rows of
2048 channels, 8 x 4096 tokens) or are generic.
"""
import math

import torch

own = False

BLOCK = 32     # tokens between two saved states of the recurrence
GROUP = 128    # values that share one scale of an 8-bit checkpoint
EPS = 1e-5


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence decoding: a token through one layer's recurrence
        dict(name="scan_step_one", op="scan_step", dtype="bf16", N=1, C=2048, gated=True, gate=True, norm=True),
        # a decode batch of 256 sequences, fp32 activations, decays given
        dict(name="scan_step_batch", op="scan_step", dtype="f32", N=256, C=2048, gated=False, gate=False, norm=False),
        # a training forward of one layer, states kept for its backward
        dict(name="scan_fwd_layer", op="scan_fwd", dtype="bf16", B=8, T=4096, C=2048, gated=True, gate=True, norm=True,
             ckpt=True),
        # prefill of one long document: few channels' chains, many tokens, a length that ends inside a block
        dict(name="scan_fwd_long", op="scan_fwd", dtype="bf16", B=1, T=32785, C=2048, gated=False, gate=False,
             norm=False, ckpt=False),
        # the training backward of one layer, its input kept in 8 bits
        dict(name="scan_bwd_layer", op="scan_bwd", dtype="bf16", B=8, T=4096, C=2048, gated=True, gate=True, norm=True,
             ckpt=True, x8=True),
        # a ragged fp32 backward of odd width that kept no states: they are computed again
        dict(name="scan_bwd_odd", op="scan_bwd", dtype="f32", B=3, T=1001, C=333, gated=False, gate=False, norm=False,
             ckpt=False, x8=False),
        # one token's layer norm while decoding
        dict(name="norm_fwd_token", op="norm_fwd", dtype="bf16", R=1, D=2048),
        # the per-head norm of the delta rule's outputs (8 x 4096 x 16 rows of 128)
        dict(name="norm_fwd_heads", op="norm_fwd", dtype="bf16", R=524288, D=128),
        # a training step through the norm before a layer: forward, then backward from the 8-bit rows
        dict(name="norm_train_layer", op="norm_train", dtype="bf16", R=32768, D=2048),
        # a backward of odd width in fp32
        dict(name="norm_bwd_odd", op="norm_bwd", dtype="f32", R=5000, D=5003),
        # an activation of one layer put away in the forward and brought back in the backward
        dict(name="ckpt8_round_layer", op="ckpt8_round", dtype="bf16", R=32768, D=2048),
        # rows that end inside a group, brought back in fp32
        dict(name="ckpt8_unpack_odd", op="ckpt8_unpack", dtype="f32", R=1111, D=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "norm_fwd", "norm_train", "norm_bwd",
                     "ckpt8_round", "ckpt8_unpack"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 1 << 25                                    # elements of one activation
    if op.startswith("scan"):
        gated = rng.random() < 0.7
        case = dict(op=op, dtype=dtype, gated=gated, gate=gated and rng.random() < 0.6, norm=gated and rng.random() < 0.6)
        C = _log_int(rng, 1, 8192)
        if rng.random() < 0.6:
            C = max(16, C // 16 * 16)
        case["C"] = C
        if op == "scan_step":
            case["N"] = _log_int(rng, 1, 1024)
            return case
        case["B"] = _log_int(rng, 1, 16)
        case["T"] = _log_int(rng, 1, max(1, min(32768, most // (C * case["B"]))))
        case["ckpt"] = rng.random() < 0.5
        if op == "scan_bwd":
            case["x8"] = rng.random() < 0.5
        return case
    D = _log_int(rng, 1, 16384)
    if rng.random() < 0.6:
        D = max(16, D // 16 * 16)
    return dict(op=op, dtype=dtype, R=_log_int(rng, 1, max(1, min(1 << 19, most // D))), D=D)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    s = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("scan"):
        C = case["C"]
        ins = (3 if case["gate"] else 2) * s if case["gated"] else s + 4       # x, decay (and gate)
        per = 2 + (10 if case["gated"] else 0) + (5 if case["gate"] else 0) + (4 if case["norm"] else 0)
        if op == "scan_step":
            n = case["N"] * C
            return {"bytes": n * (ins + s + 8) + (4 * C if case["gated"] else 0), "flops": n * per}
        B, T = case["B"], case["T"]
        n, blocks = B * T * C, B * -(-T // BLOCK) * C
        if op == "scan_fwd":
            return {"bytes": n * (ins + s) + 8 * B * C + (4 * blocks if case["ckpt"] else 0) + (4 * C if case["gated"] else 0),
                    "flops": n * per}
        xin = s if not case["x8"] else 1 + 1 / GROUP
        outs = (3 if case["gate"] else 2) * s if case["gated"] else s + 4
        return {"bytes": n * (ins - s + xin + s + outs) + 12 * B * C + (4 * blocks if case["ckpt"] else 0) +
                (8 * C if case["gated"] else 0), "flops": n * (2 * per + 10)}
    R, D = case["R"], case["D"]
    n = R * D
    if op == "norm_fwd":
        return {"bytes": n * 2 * s + 8 * D + 8 * R, "flops": 8 * n}
    if op == "norm_bwd":
        return {"bytes": n * 3 * s + 12 * D + 8 * R, "flops": 14 * n}
    codes = n + R * -(-D // GROUP)
    if op == "norm_train":   # x and dy in; y and dx out; the codes written and read; the statistics written and read
        return {"bytes": n * 4 * s + 2 * codes + 20 * D + 16 * R, "flops": 26 * n}
    if op == "ckpt8_round":
        return {"bytes": n * 2 * s + 2 * codes, "flops": 5 * n}
    return {"bytes": n * s + codes, "flops": 2 * n}


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    st = dict(case=case)
    op = case["op"]
    if op.startswith("scan"):
        C = case["C"]
        lead = (case["N"],) if op == "scan_step" else (case["B"], case["T"])
        st["x"] = normal(*lead, C)
        # channels forget over a few to a few hundred tokens
        scale = torch.exp(math.log(0.01) + (math.log(1.0) - math.log(0.01)) *
                          torch.rand(C, generator=gen, device="cuda", dtype=torch.float32))
        if case["gated"]:
            st["decay_x"], st["decay_a"] = normal(*lead, C), scale
            st["gate_x"] = normal(*lead, C) if case["gate"] else None
        else:
            alpha = torch.exp(-scale * torch.nn.functional.softplus(normal(*lead, C, dtype=torch.float32)))
            if op != "scan_step":    # a document starts: the state is left behind
                alpha[torch.rand(lead, generator=gen, device="cuda") < 1 / 1024] = 0.0
            st["alpha"] = alpha
        st["h"] = normal(lead[0], C, dtype=torch.float32)
        if op == "scan_step":
            st["h_out"] = torch.empty_like(st["h"])
        if op == "scan_bwd":
            st["grad_y"] = normal(*lead, C)
            st["grad_h"] = normal(lead[0], C, dtype=torch.float32)
            st["ckpt"] = _plain_scan(st)[2] if case["ckpt"] else None
            if case["x8"]:
                st["x8"] = _plain_pack(st.pop("x"))
        return st
    R, D = case["R"], case["D"]
    st["x"] = normal(R, D)
    if op.startswith("norm"):
        st["weight"] = 1.0 + 0.1 * normal(D, dtype=torch.float32)
        st["bias"] = 0.1 * normal(D, dtype=torch.float32)
        if op != "norm_fwd":
            st["grad_y"] = normal(R, D)
        if op == "norm_bwd":
            _, st["mean"], st["rstd"] = _plain_norm(st["x"], st["weight"], st["bias"])
    elif op == "ckpt8_unpack":
        st["x8"] = _plain_pack(st.pop("x"))
    return st


# ---------------------------------------------------------------- plain forms
def _plain_gates(case, st, x):
    """(a, v = b x, u, softplus, s, m = 1 - a^2) in 32 bits."""
    if not case["gated"]:
        return st["alpha"], x, None, None, None, None
    d = st["decay_x"].float()
    sp = torch.clamp(d, min=0) + torch.log1p(torch.exp(-torch.abs(d)))
    u = st["decay_a"] * sp
    a = torch.exp(-u)
    v, s, m = x, None, None
    if case["gate"]:
        s = 1 / (1 + torch.exp(-st["gate_x"].float()))
        v = v * s
    if case["norm"]:
        m = -torch.expm1(-2 * u)
        v = v * torch.sqrt(m)
    return a, v, u, sp, s, m


def _blocks(t, fill):
    """[B, T, C] -> [B, blocks, BLOCK, C], filled up behind the last token."""
    B, T, C = t.shape
    n = -(-T // BLOCK)
    if n * BLOCK != T:
        t = torch.cat([t, torch.full((B, n * BLOCK - T, C), fill, dtype=t.dtype, device=t.device)], 1)
    return t.reshape(B, n, BLOCK, C)


def _plain_recurrence(a, v, h0):
    """All h_t and the states before each block, from whole blocks side by side."""
    B, T, C = a.shape
    A, V = _blocks(a, 1.0), _blocks(v, 0.0)
    P, H = torch.empty_like(A), torch.empty_like(V)
    P[:, :, 0], H[:, :, 0] = A[:, :, 0], V[:, :, 0]
    for i in range(1, BLOCK):
        P[:, :, i] = A[:, :, i] * P[:, :, i - 1]
        H[:, :, i] = A[:, :, i] * H[:, :, i - 1] + V[:, :, i]
    start = torch.empty((B, A.shape[1], C), dtype=a.dtype, device=a.device)
    h = h0
    for j in range(A.shape[1]):
        start[:, j] = h
        h = P[:, j, -1] * h + H[:, j, -1]
    H += P * start[:, :, None]
    return H.reshape(B, -1, C)[:, :T], h, start


def _plain_scan(st):
    case = st["case"]
    a, v = _plain_gates(case, st, st["x"].float())[:2]
    return _plain_recurrence(a, v, st["h"])


def _plain_scan_bwd(st):
    case, dt = st["case"], _dtype(st["case"])
    x = _plain_unpack(*st["x8"]) if case["x8"] else st["x"].float()
    a, v, u, sp, s, m = _plain_gates(case, st, x)
    B, T, C = a.shape
    if case["ckpt"]:
        before = st["ckpt"]
    else:
        before = _plain_recurrence(a, v, st["h"])[2]
    A, V = _blocks(a, 1.0), _blocks(v, 0.0)
    prev = torch.empty_like(A)                      # h_{t-1}
    h = before
    for i in range(BLOCK):
        prev[:, :, i] = h
        h = A[:, :, i] * h + V[:, :, i]
    prev = prev.reshape(B, -1, C)[:, :T]
    # G_t = dy_t + a_{t+1} G_{t+1}: the same recurrence read backwards
    dy = st["grad_y"].float().clone()
    dy[:, -1] += st["grad_h"]
    shifted = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    G = _plain_recurrence(shifted.flip(1), dy.flip(1), torch.zeros_like(st["grad_h"]))[0].flip(1)
    out = {"h0": a[:, 0] * G[:, 0]}
    if not case["gated"]:
        out["x"], out["alpha"] = G.to(dt), G * prev
        return out
    b = G if s is None else G * s
    out["x"] = (b if m is None else b * torch.sqrt(m)).to(dt)
    if s is not None:
        out["gate_x"] = (G * v * (1 - s)).to(dt)
    inner = -prev
    if m is not None:
        inner = inner + torch.where(m > 0, v * a / m, torch.zeros_like(v))
    du = G * a * inner
    out["decay_x"] = (du * st["decay_a"] / (1 + torch.exp(-st["decay_x"].float()))).to(dt)
    out["decay_a"] = (du * sp).sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_norm(x, weight, bias):
    xf = x.float()
    mean = xf.mean(1)
    c = xf - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
    return (c * rstd[:, None] * weight + bias).to(x.dtype), mean, rstd


def _plain_norm_bwd(dy, x, mean, rstd, weight):
    dyf = dy.float()
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dyf * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return (dx.to(dy.dtype), (dyf * xh).sum(0, dtype=torch.float64).float(), dyf.sum(0, dtype=torch.float64).float())


def _plain_pack(x):
    lead, D = x.shape[:-1], x.shape[-1]
    n = -(-D // GROUP)
    g = torch.zeros((*lead, n * GROUP), dtype=torch.float32, device=x.device)
    g[..., :D] = x.float()
    g = g.reshape(*lead, n, GROUP)
    bits = g.abs().amax(-1).view(torch.int32)
    # the least power of two whose 448-fold holds the group's largest value
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    e = torch.clamp(e, 1, 254)
    code = (g * torch.ldexp(torch.ones((), device=x.device), 127 - e)[..., None]).to(torch.float8_e4m3fn)
    return code.reshape(*lead, n * GROUP)[..., :D].contiguous(), e.to(torch.uint8)


def _plain_unpack(code, e):
    scale = torch.ldexp(torch.ones((), device=code.device), e.int() - 127)
    return code.float() * scale.repeat_interleave(GROUP, -1)[..., :code.shape[-1]]


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(st):
    case, op, dt = st["case"], st["case"]["op"], _dtype(st["case"])
    if op == "scan_step":
        a, v = _plain_gates(case, st, st["x"].float())[:2]
        h = a * st["h"] + v
        return {"y": h.to(dt), "h": h}
    if op == "scan_fwd":
        y, h, start = _plain_scan(st)
        return {"y": y.to(dt), "h": h, "ckpt": start if case["ckpt"] else None}
    if op == "scan_bwd":
        return _plain_scan_bwd(st)
    if op == "norm_fwd":
        y, mean, rstd = _plain_norm(st["x"], st["weight"], st["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        return _plain_norm_bwd(st["grad_y"], st["x"].float(), st["mean"], st["rstd"], st["weight"])
    if op == "norm_train":
        y, mean, rstd = _plain_norm(st["x"], st["weight"], st["bias"])
        kept = _plain_pack(st["x"])
        return (y, mean, rstd) + _plain_norm_bwd(st["grad_y"], _plain_unpack(*kept), mean, rstd, st["weight"])
    if op == "ckpt8_round":
        code, e = _plain_pack(st["x"])
        return {"x": _plain_unpack(code, e).to(dt), "exponent": e}
    return {"x": _plain_unpack(*st["x8"]).to(dt)}


def _run_own(st):
    import recurrent_state_memory_amd as gdr
    case, op = st["case"], st["case"]["op"]
    if op.startswith("scan"):
        opt = dict(gate_x=st["gate_x"], normalise=case["norm"]) if case["gated"] else {}
    if op == "scan_step":
        if case["gated"]:
            y = gdr.gdr_scan_step_gated(st["h"], st["x"], st["decay_x"], st["decay_a"], h_out=st["h_out"], **opt)
        else:
            y = gdr.gdr_scan_step(st["h"], st["x"], st["alpha"], h_out=st["h_out"])
        return {"y": y, "h": st["h_out"]}
    if op == "scan_fwd":
        if case["gated"]:
            y, h, start = gdr.gdr_scan_fwd_gated(st["x"], st["decay_x"], st["decay_a"], h0=st["h"],
                                                 return_ckpt=case["ckpt"], **opt)
        else:
            y, h, start = gdr.gdr_scan_fwd(st["x"], st["alpha"], h0=st["h"], return_ckpt=case["ckpt"])
        return {"y": y, "h": h, "ckpt": start}
    if op == "scan_bwd":
        x = st["x8"] if case["x8"] else st["x"]
        kept = dict(ckpt=st["ckpt"]) if case["ckpt"] else dict(h0=st["h"])
        if case["gated"]:
            g = gdr.gdr_scan_bwd_gated(x, st["decay_x"], st["decay_a"], st["grad_y"], grad_h=st["grad_h"], **kept, **opt)
        else:
            g = gdr.gdr_scan_bwd(x, st["alpha"], st["grad_y"], grad_h=st["grad_h"], **kept)
        return g
    if op == "norm_fwd":
        y, mean, rstd, _ = gdr.gdr_norm_fwd(st["x"], st["weight"], st["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        g = gdr.gdr_norm_bwd(st["grad_y"], st["x"], st["mean"], st["rstd"], st["weight"])
        return g["x"], g["weight"], g["bias"]
    if op == "norm_train":
        y, mean, rstd, kept = gdr.gdr_norm_fwd(st["x"], st["weight"], st["bias"], eps=EPS, return_ckpt8=True)
        g = gdr.gdr_norm_bwd(st["grad_y"], kept, mean, rstd, st["weight"])
        return y, mean, rstd, g["x"], g["weight"], g["bias"]
    if op == "ckpt8_round":
        code, e = gdr.gdr_ckpt8_pack(st["x"])
        return {"x": gdr.gdr_ckpt8_unpack(code, e, dtype=_dtype(case)), "exponent": e}
    return {"x": gdr.gdr_ckpt8_unpack(*st["x8"], dtype=_dtype(case))}


# ---------------------------------------------------------------- 64 bits, from the definitions
def _value8(code, e):
    """e4m3 codes and exponents as numbers: sign, 4 bits of exponent, 3 of fraction."""
    b = code.view(torch.uint8).to(torch.int64)
    f, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(f == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((f - 7).double()))
    group = torch.arange(code.shape[-1], device=code.device) // GROUP
    return torch.where(b >= 128, -mag, mag) * torch.exp2(e.double() - 127)[..., group]


def _pack64(x):
    """The nearest e4m3 multiples of each group's scale, ties to even, and the scale's exponents."""
    R, D = x.shape
    xd = x.double()
    out, exps = torch.empty_like(xd), []
    for c0 in range(0, D, GROUP):
        g = xd[:, c0:c0 + GROUP]
        top = g.abs().amax(1)
        frac, p = torch.frexp(top / 448.0)           # top/448 = frac 2^p, frac in [1/2, 1)
        p = torch.where(frac == 0.5, p - 1, p)
        p = torch.where(top == 0, torch.full_like(p, -126), p).clamp(-126, 127)
        v = g * torch.exp2(-p.double())[:, None]
        lead = torch.frexp(v)[1] - 1
        step = torch.exp2((torch.clamp(lead, min=-6) - 3).double())
        out[:, c0:c0 + GROUP] = torch.round(v / step) * step * torch.exp2(p.double())[:, None]
        exps.append(p + 127)
    return out, torch.stack(exps, 1).to(torch.uint8)


def _norm64(x, weight, bias):
    xd = x.double()
    mean = xd.sum(1) / x.shape[1]
    var = ((xd - mean[:, None]) ** 2).sum(1) / x.shape[1]
    rstd = (var + EPS) ** -0.5
    return ((xd - mean[:, None]) * rstd[:, None]) * weight.double() + bias.double(), mean, rstd


def _norm_bwd64(dy, x, mean, rstd, weight):
    D = dy.shape[1]
    hat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    d = dy.double()
    p = d * weight.double()
    s0, s1 = p.sum(1, keepdim=True), (p * hat).sum(1, keepdim=True)
    return (rstd.double()[:, None] * (D * p - s0 - hat * s1) / D, (d * hat).sum(0), d.sum(0))


def _gates64(case, st, t):
    """a, b and their makings at token t (or for all rows of a step)."""
    if not case["gated"]:
        a = st["alpha"][:, t].double()
        return a, torch.ones_like(a), None, None, None, None
    d, scale = st["decay_x"][:, t].double(), st["decay_a"].double()
    sp = torch.logaddexp(d, torch.zeros_like(d))
    a = torch.exp(-scale * sp)
    s = torch.sigmoid(st["gate_x"][:, t].double()) if case["gate"] else torch.ones_like(a)
    n = torch.sqrt(-torch.expm1(-2 * scale * sp)) if case["norm"] else torch.ones_like(a)
    return a, s * n, d, sp, s, n


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "scan_step":
        one = {k: v[:, None] for k, v in st.items() if k in ("alpha", "decay_x", "gate_x") and v is not None}
        if case["gated"]:
            one["decay_a"] = st["decay_a"]
        a, b = _gates64(case, one, 0)[:2]
        h = a * st["h"].double() + b * st["x"].double()
        return {"y": h, "h": h}
    if op == "scan_fwd":
        T = case["T"]
        y = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
        starts, h = [], st["h"].double()
        for t in range(T):
            if t % BLOCK == 0:
                starts.append(h)
            a, b = _gates64(case, st, t)[:2]
            h = a * h + b * st["x"][:, t].double()
            y[:, t] = h
        return {"y": y, "h": h, "ckpt": torch.stack(starts, 1) if case["ckpt"] else None}
    if op == "scan_bwd":
        T = case["T"]
        x = _value8(*st["x8"]) if case["x8"] else st["x"].double()
        prev = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        h = st["h"].double()
        for t in range(T):
            if case["ckpt"] and t % BLOCK == 0:
                h = st["ckpt"][:, t // BLOCK].double()
            prev[:, t] = h
            a, b = _gates64(case, st, t)[:2]
            h = a * h + b * x[:, t]
        out = {k: torch.empty(x.shape, dtype=torch.float64, device="cuda")
               for k in (["x", "alpha"] if not case["gated"] else ["x", "decay_x"] + ["gate_x"] * case["gate"])}
        if case["gated"]:
            out["decay_a"] = torch.zeros(case["C"], dtype=torch.float64, device="cuda")
        K = st["grad_h"].double()                    # dL/dh_t from what follows t
        for t in reversed(range(T)):
            a, b, d, sp, s, n = _gates64(case, st, t)
            G = K + st["grad_y"][:, t].double()
            out["x"][:, t] = G * b
            da = G * prev[:, t]
            if case["gated"]:
                if case["gate"]:
                    out["gate_x"][:, t] = G * x[:, t] * n * s * (1 - s)
                if case["norm"]:                     # n = sqrt(1 - a^2)
                    da = da - G * x[:, t] * s * a / n
                du = -a * da
                out["decay_x"][:, t] = du * st["decay_a"].double() * torch.sigmoid(d)
                out["decay_a"] += (du * sp).sum(0)
            else:
                out["alpha"][:, t] = da
            K = a * G
        out["h0"] = K
        return out
    if op == "norm_fwd":
        y, mean, rstd = _norm64(st["x"], st["weight"], st["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        return _norm_bwd64(st["grad_y"], st["x"], st["mean"], st["rstd"], st["weight"])
    if op == "norm_train":
        y, mean, rstd = _norm64(st["x"], st["weight"], st["bias"])
        return (y, mean, rstd) + _norm_bwd64(st["grad_y"], _pack64(st["x"])[0], mean, rstd, st["weight"])
    if op == "ckpt8_round":
        v, e = _pack64(st["x"])
        return {"x": v, "exponent": e}
    return {"x": _value8(*st["x8"])}
