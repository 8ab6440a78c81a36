"""The workloads of the short causal convolution, the selective state space scan
and the gated group norm: their inputs, one pass through each operator in plain
torch and through the library, their least traffic and their 64-bit values.

Widths follow the framework's layer workload (16 heads of 128 channels: rows of
2048 channels, 8 x 4096 tokens) or are generic; 16 states a channel and four taps
are the usual sizes of such layers.
"""
import math

import torch

own = False

BLOCK = 32     # tokens between two saved states of the scan
EPS = 1e-5


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence decoding: a token through one layer's convolution
        dict(name="conv_step_one", op="conv_step", dtype="bf16", N=1, C=2048, K=4, bias=True, silu=True),
        # a training forward of one layer
        dict(name="conv_fwd_layer", op="conv_fwd", dtype="bf16", B=8, T=4096, C=2048, K=4, bias=True, silu=True,
             lens=False),
        # its backward
        dict(name="conv_bwd_layer", op="conv_bwd", dtype="bf16", B=8, T=4096, C=2048, K=4, bias=True, silu=True,
             lens=False),
        # a padded fp32 batch of odd width, three taps and no activation
        dict(name="conv_bwd_odd", op="conv_bwd", dtype="f32", B=3, T=1001, C=333, K=3, bias=False, silu=False, lens=True),
        # a decode batch of 256 sequences
        dict(name="ssm_step_batch", op="ssm_step", dtype="bf16", R=256, C=2048, N=16, G=1, D=True, z=True, bias=True,
             softplus=True),
        # a training forward of one layer, states kept for its backward
        dict(name="ssm_fwd_layer", op="ssm_fwd", dtype="bf16", B=8, T=4096, C=2048, N=16, G=1, D=True, z=True, bias=True,
             softplus=True, ckpt=True, lens=False),
        # prefill of one long document: few channels' chains, many tokens, a length that ends inside a block
        dict(name="ssm_fwd_long", op="ssm_fwd", dtype="bf16", B=1, T=32785, C=2048, N=16, G=1, D=True, z=False, bias=True,
             softplus=True, ckpt=False, lens=False),
        # the training backward of one layer
        dict(name="ssm_bwd_layer", op="ssm_bwd", dtype="bf16", B=8, T=4096, C=2048, N=16, G=1, D=True, z=True, bias=True,
             softplus=True, ckpt=True, lens=False),
        # a padded fp32 batch, three groups of odd width, eight states; it kept none of them: they are computed again
        dict(name="ssm_bwd_odd", op="ssm_bwd", dtype="f32", B=2, T=777, C=303, N=8, G=3, D=False, z=False, bias=False,
             softplus=False, ckpt=False, lens=True),
        # one token's heads, normalised and gated while decoding
        dict(name="gnorm_fwd_token", op="gnorm_fwd", dtype="bf16", R=1, C=2048, G=16, z=True, silu=True, center=False),
        # a training step through the norm and gate behind 16 heads: forward, then backward
        dict(name="gnorm_train_layer", op="gnorm_train", dtype="bf16", R=32768, C=2048, G=16, z=True, silu=True,
             center=False),
        # a backward of odd groups in fp32, mean taken off, activation on the output
        dict(name="gnorm_bwd_odd", op="gnorm_bwd", dtype="f32", R=5000, C=2331, G=7, z=False, silu=True, center=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_bwd", "ssm_step", "ssm_fwd", "ssm_fwd", "ssm_bwd", "ssm_bwd",
                     "gnorm_fwd", "gnorm_train", "gnorm_bwd"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))

    def flag(p):
        return rng.random() < p

    def width(most, least=1):
        c = _log_int(rng, least, most)
        return max(16, c // 16 * 16) if flag(0.6) else c

    most = 1 << 25                                    # elements of one activation
    if op.startswith("conv"):
        case.update(C=width(8192), K=rng.choice([2, 3, 4, 4, 4, 5, 8]), bias=flag(0.6), silu=flag(0.7))
        if op == "conv_step":
            case["N"] = _log_int(rng, 1, 1024)
            return case
        case["B"] = _log_int(rng, 1, 16)
        case["T"] = _log_int(rng, 1, max(1, min(32768, most // (case["C"] * case["B"]))))
        case["lens"] = flag(0.4)
        return case
    if op.startswith("ssm"):
        case["N"] = rng.choice([16, 16, 16, 8, 32, 64, 4, 1, rng.randint(1, 64)])
        case["G"] = rng.choice([1, 1, 1, 2, 4])
        case["C"] = width(8192 // case["G"]) * case["G"]
        case.update(D=flag(0.7), z=flag(0.5), bias=flag(0.6), softplus=flag(0.8))
        if op == "ssm_step":
            case["R"] = _log_int(rng, 1, max(1, min(1024, (1 << 25) // (case["C"] * case["N"]))))
            return case
        case["B"] = _log_int(rng, 1, 16)
        states = 1 << 29                              # channels x tokens x states
        case["T"] = _log_int(rng, 1, max(1, min(32768, most // (case["C"] * case["B"]),
                                                states // (case["C"] * case["B"] * case["N"]))))
        case.update(ckpt=flag(0.5), lens=flag(0.4))
        return case
    case["G"] = rng.choice([1, 2, 3, 8, 16, 32])
    case["C"] = case["G"] * width(16384 // case["G"], 8)
    case["R"] = _log_int(rng, 1, max(1, min(1 << 19, most // case["C"])))
    case.update(z=flag(0.6), silu=flag(0.7), center=flag(0.5))
    return case


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    s = 2 if case["dtype"] == "bf16" else 4
    op, C = case["op"], case["C"]
    if op.startswith("conv"):
        K = case["K"]
        params = 4 * C * (K + (1 if case["bias"] else 0))
        act = 5 if case["silu"] else 0
        if op == "conv_step":
            n = case["N"] * C
            return {"bytes": n * s * (2 * (K - 1) + 2) + params, "flops": n * (2 * K + act)}
        n, edge = case["B"] * case["T"] * C, case["B"] * (K - 1) * C * s
        if op == "conv_fwd":
            return {"bytes": 2 * n * s + 2 * edge + params, "flops": n * (2 * K + act)}
        return {"bytes": 3 * n * s + 3 * edge + 2 * params, "flops": n * (4 * K + (2 * K + 2 * act if case["silu"] else 0))}
    if op.startswith("ssm"):
        N, G = case["N"], case["G"]
        per_c = 12 if case["softplus"] else 1         # per channel and token, beside the states
        per_c += (2 if case["D"] else 0) + (6 if case["z"] else 0)
        params = 4 * C * (N + (1 if case["D"] else 0) + (1 if case["bias"] else 0))
        acts = 2 + (1 if case["z"] else 0)            # x, dt, z
        if op == "ssm_step":
            n = case["R"] * C
            return {"bytes": n * (s * (acts + 1) + 8 * N) + 2 * case["R"] * G * N * s + params,
                    "flops": n * (7 * N + per_c)}
        B, T = case["B"], case["T"]
        n, vec, hs = B * T * C, 2 * B * T * G * N * s, 4 * B * C * N
        blocks = 4 * B * -(-T // BLOCK) * C * N if case["ckpt"] else 0
        if op == "ssm_fwd":
            return {"bytes": n * s * (acts + 1) + vec + 2 * hs + blocks + params, "flops": n * (7 * N + per_c)}
        return {"bytes": n * s * (2 * acts + 1) + 2 * vec + hs * (2 if case["ckpt"] else 3) + blocks + 2 * params,
                "flops": n * (20 * N + 3 * per_c)}
    R, G = case["R"], case["G"]
    n = R * C
    stats = 4 * R * G * (2 if case["center"] else 1)
    acts = 2 if case["z"] else 1
    act = 5 if case["silu"] else 0
    if op == "gnorm_fwd":
        return {"bytes": n * s * (acts + 1) + 8 * C + stats, "flops": n * (7 + act)}
    if op == "gnorm_bwd":
        return {"bytes": n * s * (2 * acts + 1) + 16 * C + stats, "flops": n * (18 + 2 * act)}
    return {"bytes": n * s * (acts + 1 + 2 * acts + 1) + 24 * C + 2 * stats, "flops": n * (25 + 3 * act)}


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, op, C = _dtype(case), case["op"], case["C"]

    def normal(*shape, dtype=dt, scale=1.0):
        return (scale * torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    def lengths():
        """A padded batch: rows of any length up to T, one of them full, at times an empty one."""
        B, T = case["B"], case["T"]
        n = (uniform(B) * (T + 1)).to(torch.int32).clamp(0, T)
        n[0] = T
        return n

    f32 = torch.float32
    st = dict(case=case)
    if op.startswith("conv"):
        K = case["K"]
        lead = (case["N"],) if op == "conv_step" else (case["B"], case["T"])
        st["x"], st["state"] = normal(*lead, C), normal(lead[0], K - 1, C)
        st["weight"] = (uniform(C, K) * 2 - 1) / math.sqrt(K)
        st["bias"] = normal(C, dtype=f32, scale=0.1) if case["bias"] else None
        if op == "conv_step":
            st["state_out"] = torch.empty_like(st["state"])
            return st
        st["lens"] = lengths() if case["lens"] else None
        if op == "conv_bwd":
            st["grad_y"], st["grad_state"] = normal(*lead, C), normal(lead[0], K - 1, C)
        return st
    if op.startswith("ssm"):
        N, G = case["N"], case["G"]
        lead = (case["R"],) if op == "ssm_step" else (case["B"], case["T"])
        st["x"] = torch.nn.functional.silu(normal(*lead, C, dtype=f32)).to(dt)     # what the convolution before it gives
        # each channel's time step lies between 1e-3 and 1e-1, moved by its input
        step = torch.exp(math.log(1e-3) + math.log(1e2) * uniform(C))
        inv = step + torch.log(-torch.expm1(-step))                                # softplus^-1
        raw = normal(*lead, C, dtype=f32, scale=0.5)
        st["dt_bias"] = inv if case["bias"] else None
        if not case["bias"]:
            raw = raw + inv
        if not case["softplus"]:
            raw = step * torch.exp(raw - inv) if not case["bias"] else step * torch.exp(raw) - inv
        st["dt"] = raw.to(dt)
        # decay rates 1 ... N per unit of time step, a little different for each channel
        st["A"] = -torch.arange(1, N + 1, device="cuda", dtype=f32) * torch.exp(normal(C, N, dtype=f32, scale=0.1))
        st["B"], st["C"] = normal(*lead, G, N), normal(*lead, G, N)
        st["D"] = 1.0 + normal(C, dtype=f32, scale=0.1) if case["D"] else None
        st["z"] = normal(*lead, C) if case["z"] else None
        st["h"] = normal(lead[0], C, N, dtype=f32, scale=0.1)
        if op == "ssm_step":
            st["h_out"] = torch.empty_like(st["h"])
            return st
        st["lens"] = lengths() if case["lens"] else None
        if op == "ssm_bwd":
            st["grad_y"], st["grad_h"] = normal(*lead, C), normal(lead[0], C, N, dtype=f32, scale=0.1)
            st["ckpt"] = _plain_ssm_fwd(st)["ckpt"] if case["ckpt"] else None
        return st
    R, G = case["R"], case["G"]
    st["x"] = normal(R, C)
    st["z"] = normal(R, C) if case["z"] else None
    st["weight"], st["bias"] = 1.0 + normal(C, dtype=f32, scale=0.1), normal(C, dtype=f32, scale=0.1)
    if op != "gnorm_fwd":
        st["grad_y"] = normal(R, C)
    if op == "gnorm_bwd":
        _, st["mean"], st["rstd"] = _plain_gnorm(st)
    return st


# ---------------------------------------------------------------- plain forms
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _live(lens, T):
    """[B,T] truth values: the tokens that belong to a row."""
    return torch.arange(T, device=lens.device)[None] < lens[:, None]


def _plain_conv(st):
    """(u, the inputs with the K-1 before them) in 32 bits."""
    x = st["x"].float()
    T, K = x.shape[1], st["weight"].shape[1]
    full = torch.cat([st["state"].float(), x], 1)
    u = sum(st["weight"][:, j] * full[:, j:j + T] for j in range(K))
    return (u if st["bias"] is None else u + st["bias"]), full


def _tail(full, st):
    """The K-1 inputs before each row's end."""
    K, T = st["weight"].shape[1], st["x"].shape[1]
    if st["lens"] is None:
        return full[:, T:]
    at = st["lens"].long()[:, None] + torch.arange(K - 1, device=full.device)
    return full.gather(1, at[:, :, None].expand(-1, -1, full.shape[2]))


def _plain_conv_fwd(st):
    dt = _dtype(st["case"])
    u, full = _plain_conv(st)
    y = u * _sigmoid(u) if st["case"]["silu"] else u
    if st["lens"] is not None:
        y = torch.where(_live(st["lens"], y.shape[1])[:, :, None], y, torch.zeros_like(y))
    return {"y": y.to(dt), "state": _tail(full, st).to(dt)}


def _plain_conv_bwd(st):
    case, dt = st["case"], _dtype(st["case"])
    u, full = _plain_conv(st)
    K, T = case["K"], case["T"]
    g = st["grad_y"].float()
    if case["silu"]:
        s = _sigmoid(u)
        g = g * (s * (1 + u * (1 - s)))
    if st["lens"] is not None:
        g = torch.where(_live(st["lens"], T)[:, :, None], g, torch.zeros_like(g))
    gf = torch.zeros_like(full)
    for j in range(K):
        gf[:, j:j + T] += st["weight"][:, j] * g
    if st["lens"] is None:
        gf[:, T:] += st["grad_state"].float()
    else:
        at = st["lens"].long()[:, None] + torch.arange(K - 1, device=full.device)
        gf.scatter_add_(1, at[:, :, None].expand(-1, -1, full.shape[2]), st["grad_state"].float())
    out = {"x": gf[:, K - 1:].to(dt), "state": gf[:, :K - 1].to(dt),
           "weight": torch.stack([(g * full[:, j:j + T]).sum((0, 1), dtype=torch.float64) for j in range(K)], 1).float()}
    if case["bias"]:
        out["bias"] = g.sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_conv_step(st):
    dt = _dtype(st["case"])
    full = torch.cat([st["state"].float(), st["x"].float()[:, None]], 1)
    u = sum(st["weight"][:, j] * full[:, j] for j in range(full.shape[1]))
    if st["bias"] is not None:
        u = u + st["bias"]
    y = u * _sigmoid(u) if st["case"]["silu"] else u
    return {"y": y.to(dt), "state": full[:, 1:].to(dt)}


def _time_step(st):
    """(Delta, its pre-activation) in 32 bits."""
    d = st["dt"].float()
    if st["dt_bias"] is not None:
        d = d + st["dt_bias"]
    if not st["case"]["softplus"]:
        return d, d
    return torch.clamp(d, min=0) + torch.log1p(torch.exp(-torch.abs(d))), d


def _spread(v, C):
    """[..., G, N] -> [..., C, N]: each group's vector for each of its channels."""
    G, N = v.shape[-2:]
    return v.float()[..., :, None, :].expand(*v.shape[:-2], G, C // G, N).reshape(*v.shape[:-2], C, N)


def _blocks(t, fill):
    """[B, T, ...] -> [B, blocks, BLOCK, ...], filled up behind the last token."""
    B, T = t.shape[:2]
    n = -(-T // BLOCK)
    if n * BLOCK != T:
        t = torch.cat([t, torch.full((B, n * BLOCK - T, *t.shape[2:]), fill, dtype=t.dtype, device=t.device)], 1)
    return t.reshape(B, n, BLOCK, *t.shape[2:])


def _plain_recurrence(a, v, h0):
    """All h_t = a_t h_{t-1} + v_t, the last one and the ones before each block, from whole blocks side by side."""
    B, T = a.shape[:2]
    A, H = _blocks(a, 1.0).clone(), _blocks(v, 0.0).clone()
    for i in range(1, BLOCK):
        H[:, :, i] += A[:, :, i] * H[:, :, i - 1]
        A[:, :, i] *= A[:, :, i - 1]
    start = torch.empty((B, A.shape[1], *a.shape[2:]), dtype=a.dtype, device=a.device)
    h = h0
    for j in range(A.shape[1]):
        start[:, j] = h
        h = A[:, j, -1] * h + H[:, j, -1]
    H += A * start[:, :, None]
    return H.reshape(B, -1, *a.shape[2:])[:, :T], h, start


def _plain_ssm(st):
    """(x, Delta, its pre-activation, decays, v) in 32 bits, tokens behind a row's end without effect."""
    x = st["x"].float()
    delta, pre = _time_step(st)
    if st["lens"] is not None:
        live = _live(st["lens"], x.shape[1])[:, :, None]
        x, delta = torch.where(live, x, 0.0), torch.where(live, delta, 0.0)
    a = torch.exp(delta[..., None] * st["A"])
    return x, delta, pre, a, (delta * x)[..., None] * _spread(st["B"], x.shape[2])


def _plain_ssm_fwd(st):
    case, dt = st["case"], _dtype(st["case"])
    x, _, _, a, v = _plain_ssm(st)
    h, last, start = _plain_recurrence(a, v, st["h"])
    y = (h * _spread(st["C"], x.shape[2])).sum(-1)
    if case["D"]:
        y = y + st["D"] * x
    if case["z"]:
        z = st["z"].float()
        y = y * z * _sigmoid(z)
    if st["lens"] is not None:
        y = torch.where(_live(st["lens"], x.shape[1])[:, :, None], y, 0.0)
    return {"y": y.to(dt), "h": last, "ckpt": start.transpose(2, 3).contiguous() if case["ckpt"] else None}


def _plain_ssm_bwd(st):
    case, dt = st["case"], _dtype(st["case"])
    x, delta, pre, a, v = _plain_ssm(st)
    B, T, C = x.shape
    G, N = case["G"], case["N"]
    if case["ckpt"]:
        start = st["ckpt"].transpose(2, 3)
    else:
        start = _plain_recurrence(a, v, st["h"])[2]
    a_, v_ = _blocks(a, 1.0), _blocks(v, 0.0)
    prev = torch.empty_like(a_)                     # h_{t-1}
    h = start
    for i in range(BLOCK):
        prev[:, :, i] = h
        h = a_[:, :, i] * h + v_[:, :, i]
    prev = prev.reshape(B, -1, C, N)[:, :T]
    h = a * prev + v
    del a_, v_, v
    live = None if st["lens"] is None else _live(st["lens"], T)[:, :, None]
    g = st["grad_y"].float()
    if live is not None:
        g = torch.where(live, g, 0.0)
    out = {}
    Cs = _spread(st["C"], C)
    if case["z"]:
        z = st["z"].float()
        s = _sigmoid(z)
        u = (h * Cs).sum(-1)
        if case["D"]:
            u = u + st["D"] * x
        gz = g * u * s * (1 + z * (1 - s))
        out["z"] = (gz if live is None else torch.where(live, gz, 0.0)).to(dt)
        g = g * z * s
    out["C"] = (g[..., None] * h).reshape(B, T, G, C // G, N).sum(3).to(dt)
    # H_t = C_t g_t + a_{t+1} H_{t+1}: the same recurrence read backwards
    drive = g[..., None] * Cs
    drive[:, -1] += st["grad_h"]
    shifted = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    H = _plain_recurrence(shifted.flip(1), drive.flip(1), torch.zeros_like(st["grad_h"]))[0].flip(1)
    del drive, shifted, h
    out["h0"] = a[:, 0] * H[:, 0]
    p = (H * _spread(st["B"], C)).sum(-1)
    out["B"] = (H * (delta * x)[..., None]).reshape(B, T, G, C // G, N).sum(3).to(dt)
    q = H * a * prev
    out["A"] = (q * delta[..., None]).sum((0, 1), dtype=torch.float64).float()
    dd = (q * st["A"]).sum(-1) + p * x
    if case["softplus"]:
        dd = dd * _sigmoid(pre)
    if live is not None:
        dd = torch.where(live, dd, 0.0)
    dx = p * delta
    if case["D"]:
        dx = dx + st["D"] * g
        out["D"] = (g * x).sum((0, 1), dtype=torch.float64).float()
    out["x"] = dx.to(dt)
    out["dt"] = dd.to(dt)
    if case["bias"]:
        out["dt_bias"] = dd.sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_ssm_step(st):
    case, dt = st["case"], _dtype(st["case"])
    x, C = st["x"].float(), case["C"]
    delta = _time_step(st)[0]
    h = torch.exp(delta[..., None] * st["A"]) * st["h"] + (delta * x)[..., None] * _spread(st["B"], C)
    y = (h * _spread(st["C"], C)).sum(-1)
    if case["D"]:
        y = y + st["D"] * x
    if case["z"]:
        z = st["z"].float()
        y = y * z * _sigmoid(z)
    return {"y": y.to(dt), "h": h}


def _plain_gnorm(st):
    case = st["case"]
    R, C, G = case["R"], case["C"], case["G"]
    x = st["x"].float().reshape(R, G, C // G)
    mean = None
    if case["center"]:
        mean = x.mean(2)
        x = x - mean[:, :, None]
    rstd = 1 / torch.sqrt((x * x).mean(2) + EPS)
    u = (x * rstd[:, :, None]).reshape(R, C) * st["weight"] + st["bias"]
    if case["z"]:
        z = st["z"].float()
        y = u * z * _sigmoid(z) if case["silu"] else u * z
    else:
        y = u * _sigmoid(u) if case["silu"] else u
    return y.to(st["x"].dtype), mean, rstd


def _plain_gnorm_bwd(st, mean, rstd):
    case, dt = st["case"], _dtype(st["case"])
    R, C, G = case["R"], case["C"], case["G"]
    x = st["x"].float().reshape(R, G, C // G)
    if case["center"]:
        x = x - mean[:, :, None]
    xh = x * rstd[:, :, None]
    u = xh.reshape(R, C) * st["weight"] + st["bias"]
    g = st["grad_y"].float()
    out = {}
    if case["z"]:
        z = st["z"].float()
        if case["silu"]:
            s = _sigmoid(z)
            out["z"] = (g * u * s * (1 + z * (1 - s))).to(dt)
            g = g * z * s
        else:
            out["z"] = (g * u).to(dt)
            g = g * z
    elif case["silu"]:
        s = _sigmoid(u)
        g = g * s * (1 + u * (1 - s))
    out["weight"] = (g * xh.reshape(R, C)).sum(0, dtype=torch.float64).float()
    out["bias"] = g.sum(0, dtype=torch.float64).float()
    g = (g * st["weight"]).reshape(R, G, C // G)
    dx = g - xh * (g * xh).mean(2, keepdim=True)
    if case["center"]:
        dx = dx - g.mean(2, keepdim=True)
    out["x"] = (dx * rstd[:, :, None]).reshape(R, C).to(dt)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(st):
    op = st["case"]["op"]
    if op == "gnorm_bwd":
        return _plain_gnorm_bwd(st, st["mean"], st["rstd"])
    if op.startswith("gnorm"):
        y, mean, rstd = _plain_gnorm(st)
        out = {"y": y, "mean": mean, "rstd": rstd}
        if op == "gnorm_train":
            out["grads"] = _plain_gnorm_bwd(st, mean, rstd)
        return out
    return {"conv_step": _plain_conv_step, "conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd,
            "ssm_step": _plain_ssm_step, "ssm_fwd": _plain_ssm_fwd, "ssm_bwd": _plain_ssm_bwd}[op](st)


def _run_own(st):
    import recurrent_state_memory_amd as gdr
    case, op = st["case"], st["case"]["op"]
    if op == "conv_step":
        y = gdr.gdr_conv_step(st["state"], st["x"], st["weight"], st["bias"], silu=case["silu"],
                              state_out=st["state_out"])
        return {"y": y, "state": st["state_out"]}
    if op == "conv_fwd":
        y, state = gdr.gdr_conv_fwd(st["x"], st["weight"], st["bias"], state=st["state"], lens=st["lens"],
                                    silu=case["silu"])
        return {"y": y, "state": state}
    if op == "conv_bwd":
        return gdr.gdr_conv_bwd(st["grad_y"], st["x"], st["weight"], st["bias"], state=st["state"], lens=st["lens"],
                                silu=case["silu"], grad_state=st["grad_state"])
    if op.startswith("ssm"):
        opt = dict(D=st["D"], z=st["z"], dt_bias=st["dt_bias"], softplus=case["softplus"])
        ins = st["x"], st["dt"], st["A"], st["B"], st["C"]
    if op == "ssm_step":
        y = gdr.gdr_ssm_step(st["h"], *ins, h_out=st["h_out"], **opt)
        return {"y": y, "h": st["h_out"]}
    if op == "ssm_fwd":
        y, h, ckpt = gdr.gdr_ssm_fwd(*ins, h0=st["h"], lens=st["lens"], return_ckpt=case["ckpt"], **opt)
        return {"y": y, "h": h, "ckpt": ckpt}
    if op == "ssm_bwd":
        kept = dict(ckpt=st["ckpt"]) if case["ckpt"] else dict(h0=st["h"])
        return gdr.gdr_ssm_bwd(st["grad_y"], *ins, lens=st["lens"], grad_h=st["grad_h"], **kept, **opt)
    opt = dict(z=st["z"], silu=case["silu"])
    if op == "gnorm_bwd":
        return gdr.gdr_gnorm_bwd(st["grad_y"], st["x"], st["mean"], st["rstd"], case["G"], st["weight"], st["bias"], **opt)
    y, mean, rstd = gdr.gdr_gnorm_fwd(st["x"], case["G"], st["weight"], st["bias"], center=case["center"], eps=EPS, **opt)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if op == "gnorm_train":
        out["grads"] = gdr.gdr_gnorm_bwd(st["grad_y"], st["x"], mean, rstd, case["G"], st["weight"], st["bias"], **opt)
    return out


# ---------------------------------------------------------------- 64 bits, from the definitions
def _act64(v):
    """silu and its slope."""
    s = torch.sigmoid(v)
    return v * s, s + v * s * torch.sigmoid(-v)


def _conv64(st, grads):
    case = st["case"]
    K, T, C = case["K"], case["T"], case["C"]
    w = st["weight"].double()
    rows = torch.cat([st["state"], st["x"]], 1).double()
    u = (rows.unfold(1, K, 1) * w).sum(-1)
    if case["bias"]:
        u = u + st["bias"].double()
    y, slope = _act64(u) if case["silu"] else (u, torch.ones_like(u))
    ends = [T] * case["B"] if st["lens"] is None else st["lens"].tolist()
    if not grads:
        for b, e in enumerate(ends):
            y[b, e:] = 0
        return {"y": y, "state": torch.stack([rows[b, e:e + K - 1] for b, e in enumerate(ends)])}
    du = st["grad_y"].double() * slope
    grow = torch.zeros_like(rows)
    gw = torch.zeros((C, K), dtype=torch.float64, device="cuda")
    gb = torch.zeros(C, dtype=torch.float64, device="cuda")
    for b, e in enumerate(ends):
        grow[b, e:e + K - 1] = st["grad_state"][b].double()
        d = du[b, :e]
        gb += d.sum(0)
        for j in range(K):
            grow[b, j:j + e] += d * w[:, j]
            gw[:, j] += (d * rows[b, j:j + e]).sum(0)
    # what a row's tail takes from behind its last token belongs to no input
    out = {"x": grow[:, K - 1:], "state": grow[:, :K - 1], "weight": gw}
    if case["bias"]:
        out["bias"] = gb
    return out


def _token64(st, t):
    """(Delta, its slope, a, x, B, C) at token t, or of all rows of a step (t = None)."""
    case = st["case"]

    def at(name):
        v = st[name]
        return (v if t is None else v[:, t]).double()
    pre = at("dt") + (st["dt_bias"].double() if case["bias"] else 0.0)
    delta, slope = pre, torch.ones_like(pre)
    if case["softplus"]:
        delta, slope = torch.logaddexp(pre, torch.zeros_like(pre)), torch.sigmoid(pre)
    each = case["C"] // case["G"]
    a = torch.exp(torch.einsum("bc,cn->bcn", delta, st["A"].double()))
    return (delta, slope, a, at("x"), at("B").repeat_interleave(each, 1), at("C").repeat_interleave(each, 1))


def _ssm_step64(st):
    case = st["case"]
    delta, _, a, x, Bv, Cv = _token64(st, None)
    h = a * st["h"].double() + Bv * (delta * x)[:, :, None]
    y = (Cv * h).sum(2)
    if case["D"]:
        y = y + st["D"].double() * x
    if case["z"]:
        y = y * _act64(st["z"].double())[0]
    return {"y": y, "h": h}


def _ssm_fwd64(st):
    case = st["case"]
    y = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
    starts, h = [], st["h"].double()
    for t in range(case["T"]):
        if t % BLOCK == 0:
            starts.append(h.transpose(1, 2))
        delta, _, a, x, Bv, Cv = _token64(st, t)
        new = a * h + Bv * (delta * x)[:, :, None]
        u = (Cv * new).sum(2)
        if case["D"]:
            u = u + st["D"].double() * x
        if case["z"]:
            u = u * _act64(st["z"][:, t].double())[0]
        if st["lens"] is not None:
            on = t < st["lens"]
            new = torch.where(on[:, None, None], new, h)
            u = torch.where(on[:, None], u, 0.0)
        h = new
        y[:, t] = u
    return {"y": y, "h": h, "ckpt": torch.stack(starts, 1) if case["ckpt"] else None}


def _ssm_bwd64(st):
    case = st["case"]
    T, C, N, G = case["T"], case["C"], case["N"], case["G"]
    f64 = torch.float64
    h = st["h"].double()
    prev = torch.empty((T, *h.shape), dtype=f64, device="cuda")
    for t in range(T):
        if case["ckpt"] and t % BLOCK == 0:
            h = st["ckpt"][:, t // BLOCK].double().transpose(1, 2)
        prev[t] = h
        delta, _, a, x, Bv, _ = _token64(st, t)
        new = a * h + Bv * (delta * x)[:, :, None]
        h = new if st["lens"] is None else torch.where((t < st["lens"])[:, None, None], new, h)
    out = {k: torch.zeros(st[k].shape, dtype=f64, device="cuda")
           for k in ["x", "dt", "B", "C"] + ["z"] * case["z"]}
    out["A"] = torch.zeros((C, N), dtype=f64, device="cuda")
    if case["D"]:
        out["D"] = torch.zeros(C, dtype=f64, device="cuda")
    if case["bias"]:
        out["dt_bias"] = torch.zeros(C, dtype=f64, device="cuda")
    K = st["grad_h"].double()                        # dL/dh_t from what follows t
    for t in reversed(range(T)):
        delta, slope, a, x, Bv, Cv = _token64(st, t)
        on = None if st["lens"] is None else (t < st["lens"])
        h = a * prev[t] + Bv * (delta * x)[:, :, None]
        g = st["grad_y"][:, t].double()
        if on is not None:
            g = torch.where(on[:, None], g, 0.0)
        if case["z"]:
            value, dv = _act64(st["z"][:, t].double())
            u = (Cv * h).sum(2) + (st["D"].double() * x if case["D"] else 0.0)
            out["z"][:, t] = g * u * dv
            g = g * value
        out["C"][:, t] = (g[:, :, None] * h).reshape(-1, G, C // G, N).sum(2)
        H = K + Cv * g[:, :, None]
        if on is not None:                           # behind the end: nothing but the state passes
            H = torch.where(on[:, None, None], H, 0.0)
        out["B"][:, t] = (H * (delta * x)[:, :, None]).reshape(-1, G, C // G, N).sum(2)
        into = (H * Bv).sum(2)
        da = H * prev[t] * a
        out["A"] += (da * delta[:, :, None]).sum(0)
        ddt = ((da * st["A"].double()).sum(2) + into * x) * slope
        out["dt"][:, t] = ddt
        out["x"][:, t] = into * delta
        if case["bias"]:
            out["dt_bias"] += ddt.sum(0)
        if case["D"]:
            out["x"][:, t] += st["D"].double() * g
            out["D"] += (g * x).sum(0)
        K = a * H if on is None else torch.where(on[:, None, None], a * H, K)
    out["h0"] = K
    return out


def _gnorm64(st, mean=None, rstd=None, grads=False):
    case = st["case"]
    R, C, G = case["R"], case["C"], case["G"]
    x = st["x"].double().view(R, G, -1)
    if rstd is None:
        mean = x.sum(-1) / x.shape[-1] if case["center"] else None
        c = x - mean.unsqueeze(-1) if case["center"] else x
        rstd = ((c ** 2).sum(-1) / x.shape[-1] + EPS) ** -0.5
    else:
        mean, rstd = (None if mean is None else mean.double()), rstd.double()
        c = x - mean.unsqueeze(-1) if case["center"] else x
    hat = c * rstd.unsqueeze(-1)
    w, b = st["weight"].double(), st["bias"].double()
    u = hat.view(R, C) * w + b
    z = st["z"].double() if case["z"] else None
    gate, slope = (None, None) if z is None else _act64(z) if case["silu"] else (z, torch.ones_like(z))
    if not grads:
        y = u * gate if case["z"] else _act64(u)[0] if case["silu"] else u
        return y, mean, rstd
    dy = st["grad_y"].double()
    out = {}
    if case["z"]:
        out["z"], du = dy * u * slope, dy * gate
    else:
        du = dy * _act64(u)[1] if case["silu"] else dy
    out["weight"], out["bias"] = (du * hat.view(R, C)).sum(0), du.sum(0)
    p, n = (du * w).view(R, G, -1), C // G
    s1 = (p * hat).sum(-1, keepdim=True)
    s0 = p.sum(-1, keepdim=True) if case["center"] else 0.0
    out["x"] = (rstd.unsqueeze(-1) * (n * p - s0 - hat * s1) / n).view(R, C)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "conv_step":
        rows = torch.cat([st["state"], st["x"][:, None]], 1).double()
        u = (rows * st["weight"].double().t()).sum(1) + (st["bias"].double() if case["bias"] else 0.0)
        return {"y": _act64(u)[0] if case["silu"] else u, "state": rows[:, 1:]}
    if op.startswith("conv"):
        return _conv64(st, op == "conv_bwd")
    if op == "ssm_step":
        return _ssm_step64(st)
    if op == "ssm_fwd":
        return _ssm_fwd64(st)
    if op == "ssm_bwd":
        return _ssm_bwd64(st)
    if op == "gnorm_bwd":
        return _gnorm64(st, st["mean"], st["rstd"], grads=True)
    y, mean, rstd = _gnorm64(st)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if op == "gnorm_train":
        out["grads"] = _gnorm64(st, grads=True)
    return out
