"""What is measured of the selective state-space layer's operators: the short
causal convolution, the selective scan and the norms around a block fused with
its gate and residual scale.

Every case names one operator and one way of using it: over whole prompts, in
a training step (forward and gradient), or for one token per sequence.  Where
``own`` is false ``run`` computes the operator from elementary torch
operations in 32 bits; where it is true it makes the library's calls.

Sizes are those of this repository's workloads (1024 and 2048 channels, 8 x
2048 and 1 x 16384 tokens, 32768 packed tokens in 21 sequences, 256 decoding
sequences, model width 2048) with the usual 16 states a channel, and generic
ones: an inner width of twice the model's, larger states, odd widths.
"""
import math
import random

import torch

own = False
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    bf, fp = "bf16", "fp32"
    return [
        # the whole prompts of a packed batch, as a server or an evaluation runs them
        scan("scan_prompts_packed", seqs=21, tokens=32768, packed=True, D=2048, N=16, G=1, dtype=bf, z=True, init=False),
        # one long document continued from a stored state: few channels' worth of parallel work
        scan("scan_long_prompt", seqs=1, tokens=16384, D=2048, N=16, G=1, dtype=bf, z=True, init=True),
        # a training step of the layer at 8 x 2048 tokens
        scan("scan_train_step", seqs=8, tokens=16384, D=2048, N=16, G=1, dtype=bf, z=True, init=False, train=True),
        # ragged training in fp32 with a larger state, two groups of B and C and an odd width
        scan("scan_train_wide_state_ragged", seqs=5, tokens=1531, packed=True, D=330, N=64, G=2, dtype=fp, z=False, init=True, train=True),
        # a short prompt of a small model in fp32: latency
        scan("scan_short_prompt", seqs=1, tokens=256, D=128, N=16, G=1, dtype=fp, z=False, init=False),
        # one token for each of 256 decoding sequences
        dict(name="scan_decode", op="scan_step", seqs=256, D=2048, N=16, G=1, dtype=bf, z=True),
        # the convolution before the scan, over packed prompts and in a training step
        dict(name="conv_prompts_packed", op="conv", seqs=21, tokens=32768, packed=True, D=2048, W=4, dtype=bf, bias=True, act=True, init=False, train=False),
        dict(name="conv_train_step", op="conv", seqs=8, tokens=16384, packed=False, D=4096, W=4, dtype=bf, bias=True, act=True, init=False, train=True),
        # one token for each of 256 decoding sequences: latency
        dict(name="conv_decode", op="conv_step", seqs=256, D=2048, W=4, dtype=bf, bias=True, act=True),
        # the end of one block and the start of the next: prompts, a training step, decoding rows of an odd width
        dict(name="norm_prompts", op="norm", rows=32768, D=2048, dtype=bf, gate="none", post=True, pre=True, scale=True, train=False),
        dict(name="norm_gated_train_step", op="norm", rows=16384, D=2048, dtype=bf, gate="sigmoid", post=True, pre=True, scale=True, train=True),
        dict(name="norm_decode_odd_width", op="norm", rows=64, D=1001, dtype=fp, gate="silu", post=True, pre=True, scale=True, train=False),
    ]


def scan(name, *, seqs, tokens, D, N, G, dtype, z, init, packed=False, train=False):
    return dict(name=name, op="scan", seqs=seqs, tokens=tokens, packed=packed, D=D, N=N, G=G, dtype=dtype, z=z, init=init, train=train)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "scan_step", "conv", "conv", "conv_step", "norm", "norm"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op in ("scan", "scan_step"):
        c["N"] = rng.choice([4, 8, 16, 16, 16, 24, 32, 64, 128])
        c["G"] = rng.choice([1, 1, 1, 2, 4])
        c["D"] = c["G"] * _log_int(rng, 64, 4096 // c["G"])
        c["z"] = rng.random() < 0.6
    if op == "scan_step":
        c["seqs"] = _log_int(rng, 1, max(1, min(1024, (1 << 23) // (c["D"] * c["N"]))))
    elif op == "scan":
        c["train"] = rng.random() < 0.5
        c["init"] = rng.random() < 0.5
        c["packed"] = rng.random() < 0.5
        most = min(32768, (1 << (28 if c["train"] else 29)) // (c["D"] * c["N"]))
        if c["packed"]:
            c["tokens"] = _log_int(rng, 16, max(16, most))
            c["seqs"] = rng.randint(1, min(32, c["tokens"]))
        else:
            c["seqs"] = _log_int(rng, 1, 16)
            c["tokens"] = c["seqs"] * _log_int(rng, 1, max(1, most // c["seqs"]))
    elif op == "conv_step":
        c.update(seqs=_log_int(rng, 1, 1024), D=_log_int(rng, 64, 8192), W=rng.choice([2, 3, 4]), bias=rng.random() < 0.7, act=rng.random() < 0.8)
    elif op == "conv":
        c.update(D=_log_int(rng, 64, 8192), W=rng.choice([2, 3, 4]), bias=rng.random() < 0.7, act=rng.random() < 0.8, init=rng.random() < 0.5, packed=rng.random() < 0.5, train=rng.random() < 0.5)
        most = min(32768, (1 << 25) // c["D"])
        c["seqs"] = rng.randint(1, 16)
        c["tokens"] = c["seqs"] * _log_int(rng, 1, max(1, most // c["seqs"]))
    else:
        c.update(D=_log_int(rng, 64, 8192), gate=rng.choice(["none", "sigmoid", "silu"]), post=rng.random() < 0.8, pre=rng.random() < 0.8, scale=rng.random() < 0.7, train=rng.random() < 0.5)
        c["rows"] = _log_int(rng, 1, min(32768, (1 << 25) // c["D"]))
    return c


# ----------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case, seed):
    """Tokens of each sequence: equal, or ragged ones that add up."""
    n, total = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [total // n] * n
    rng = random.Random(seed * 7 + 3)
    share = [rng.uniform(0.2, 1.8) for _ in range(n)]
    lens = [int(total * s / sum(share)) for s in share]
    lens[-1] += total - sum(lens)
    return lens


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = _dtype(case)

    def randn(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        R, D = case["rows"], case["D"]
        s["y"], s["x"] = randn(R, D, dtype=dt), randn(R, D, std=2.0, dtype=dt)
        s["gate"] = randn(R, D, dtype=dt) if case["gate"] != "none" else None
        s["w_post"] = randn(D, std=0.2, mean=1.0) if case["post"] else None
        s["w_pre"] = randn(D, std=0.2, mean=1.0) if case["pre"] else None
        s["scale"] = randn(D, std=0.1, mean=0.3) if case["scale"] else None
        if case["train"]:
            s["dx_out"], s["dh"] = randn(R, D, dtype=dt), randn(R, D, dtype=dt) if case["pre"] else None
        return s
    D, step = case["D"], case["op"].endswith("_step")
    if step:
        L = n = case["seqs"]
        lead = (n,)
    else:
        lens = _lengths(case, seed)
        L, n = case["tokens"], case["seqs"]
        s["lens"] = lens
        lead = (1, L) if case["packed"] else (n, L // n)
        ends = torch.tensor(lens).cumsum(0)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).to(DEV) if case["packed"] else None
        # which sequence each token is in, and where that sequence starts
        s["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(lens)).to(DEV)
        s["start"] = torch.repeat_interleave(ends - torch.tensor(lens), torch.tensor(lens)).to(DEV)
        s["first"], s["end"] = (ends - torch.tensor(lens)).to(DEV), ends.to(DEV)
    # the input projection gives the convolution's (or scan's) input and the gate side by side
    xz = randn(*lead, 2 * D, dtype=dt)
    s["x"] = xz[..., :D]
    if case["op"].startswith("conv"):
        W = case["W"]
        s["w"] = randn(D, W, std=0.5)
        s["bias"] = randn(D, std=0.2) if case["bias"] else None
        s["state"] = randn(n, W - 1, D, dtype=dt) if step or case["init"] else None
        if step:
            s["state_out"] = torch.empty_like(s["state"])
        elif case["train"]:
            s["dy"] = randn(*lead, D, dtype=dt)
        return s
    N, G = case["N"], case["G"]
    s["z"] = xz[..., D:] if case["z"] else None
    # B and C come out of one projection; step sizes from 1e-3 to 1e-1, decays -1 .. -N
    bc = randn(*lead, 2 * G * N, dtype=dt)
    s["Bm"], s["Cm"] = (t.unflatten(-1, (G, N)) for t in bc.split(G * N, dim=-1))
    s["dt"] = randn(*lead, D, std=0.5, dtype=dt)
    size = torch.exp(torch.rand(D, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = size + torch.log(-torch.expm1(-size))
    s["A"] = -torch.arange(1, N + 1, device=DEV, dtype=torch.float32) * torch.exp(randn(D, N, std=0.1))
    s["D_skip"] = randn(D, std=0.2, mean=1.0)
    s["h"] = randn(n, D, N, std=0.5) if step or case["init"] else None
    if step:
        s["h_out"] = torch.empty_like(s["h"])
    elif case["train"]:
        s["dy"], s["dh_T"] = randn(*lead, D, dtype=dt), randn(n, D, N, std=0.1)
    return s


# ------------------------------------------------------- the library's calls

def _run_own(s):
    import momentum_delta_rule_gb300 as mdn
    c = s["case"]
    if c["op"] == "norm":
        gate = dict(gate=s["gate"], gate_act=c["gate"]) if s["gate"] is not None else {}
        kw = dict(w_post=s["w_post"], w_pre=s["w_pre"], scale=s["scale"], eps=EPS, **gate)
        if not c["train"]:
            return mdn.norm_residual_fwd(s["y"], s["x"], **kw)
        x_out, h, stats = mdn.norm_residual_fwd(s["y"], s["x"], return_stats=True, **kw)
        return x_out, h, mdn.norm_residual_bwd(s["y"], s["x"], stats, s["dx_out"], dh=s["dh"], **kw)
    if c["op"].startswith("conv"):
        kw = dict(bias=s["bias"], activation="silu" if c["act"] else None)
        if c["op"] == "conv_step":
            return mdn.short_conv_step(s["x"], s["w"], s["state"], state_out=s["state_out"], **kw), s["state_out"]
        kw.update(state=s["state"], cu_seqlens=s["cu"])
        out = mdn.short_conv_fwd(s["x"], s["w"], output_final_state=True, **kw)
        if not c["train"]:
            return out
        return out, mdn.short_conv_bwd(s["x"], s["w"], s["dy"], **kw)
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    kw = dict(D_skip=s["D_skip"], z=s["z"], dt_bias=s["dt_bias"], softplus=True)
    if c["op"] == "scan_step":
        return mdn.ssm_scan_step(*args, s["h"], h_out=s["h_out"], **kw), s["h_out"]
    kw["cu_seqlens"] = s["cu"]
    if not c["train"]:
        return mdn.ssm_scan_fwd(*args, h0=s["h"], **kw)
    y, h_T, h_chunks = mdn.ssm_scan_fwd(*args, h0=s["h"], return_chunk_states=True, **kw)
    return y, h_T, mdn.ssm_scan_bwd(*args, h_chunks, s["dy"], dh_T=s["dh_T"], need_dh0=c["init"], **kw)


# ------------------------------------------------------------ plain forms

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _norm_plain(s):
    c, dt = s["case"], _dtype(s["case"])
    y, x = s["y"].float(), s["x"].float()
    D = y.shape[1]
    w1 = s["w_post"]
    r1 = torch.rsqrt((y * y).sum(1, keepdim=True) / D + EPS) if w1 is not None else None
    n1 = y * r1 * w1 if w1 is not None else y
    if s["gate"] is not None:
        g = s["gate"].float()
        sg = _sigmoid(g)
        act, dact = (sg, sg * (1 - sg)) if c["gate"] == "sigmoid" else (g * sg, sg * (1 + g * (1 - sg)))
        b = n1 * act
    else:
        b = n1
    X = x + b * s["scale"] if s["scale"] is not None else x + b
    w2 = s["w_pre"]
    r2 = torch.rsqrt((X * X).sum(1, keepdim=True) / D + EPS) if w2 is not None else None
    h = (X * r2 * w2).to(dt) if w2 is not None else None
    if not c["train"]:
        return X.to(dt), h
    dX = s["dx_out"].float()
    out = dict.fromkeys(("dy", "dx", "dgate", "dw_post", "dw_pre", "dscale"))
    if w2 is not None:
        dh = s["dh"].float()
        out["dw_pre"] = (dh * X * r2).sum(0)
        dX = dX + r2 * w2 * dh - X * (r2 * r2 * r2) * ((dh * w2 * X).sum(1, keepdim=True) / D)
    out["dx"] = dX.to(dt)
    db = dX
    if s["scale"] is not None:
        out["dscale"] = (dX * b).sum(0)
        db = dX * s["scale"]
    if s["gate"] is not None:
        out["dgate"] = (db * n1 * dact).to(dt)
        db = db * act
    if w1 is not None:
        out["dw_post"] = (db * y * r1).sum(0)
        db = r1 * w1 * db - y * (r1 * r1 * r1) * ((db * w1 * y).sum(1, keepdim=True) / D)
    out["dy"] = db.to(dt)
    return X.to(dt), h, out


def _conv_plain(s):
    c, dt = s["case"], _dtype(s["case"])
    W, w, x = c["W"], s["w"], s["x"].reshape(-1, c["D"]).float()
    L, n = x.shape[0], len(s["lens"])
    old = n * (W - 1)
    state = s["state"].float().reshape(old, -1) if s["state"] is not None else x.new_zeros(old, x.shape[1])
    ext = torch.cat([state, x])
    t = torch.arange(L, device=x.device)
    back = torch.arange(W - 1, -1, -1, device=x.device)
    at = t[:, None] - back                       # tap j reads W - 1 - j tokens back
    at = torch.where(at >= s["start"][:, None], old + at, s["seq"][:, None] * (W - 1) + (W - 1) + at - s["start"][:, None])
    pre = ext[at[:, 0]] * w[:, 0]
    for j in range(1, W):
        pre = pre + ext[at[:, j]] * w[:, j]
    if s["bias"] is not None:
        pre = pre + s["bias"]
    sg = _sigmoid(pre)
    y = pre * sg if c["act"] else pre
    q = torch.arange(W - 1, device=x.device)
    last = s["end"][:, None] - (W - 1) + q
    last = torch.where(last >= s["first"][:, None], old + last, torch.arange(n, device=x.device)[:, None] * (W - 1) + (W - 1) + last - s["first"][:, None])
    fwd = y.to(dt).reshape(s["x"].shape), ext[last].to(dt)
    if not c["train"]:
        return fwd
    d = s["dy"].reshape(L, -1).float()
    if c["act"]:
        d = d * sg * (1 + pre * (1 - sg))
    dext = torch.zeros_like(ext)
    for j in range(W):
        dext.index_add_(0, at[:, j], d * w[:, j])
    dw = torch.stack([(d * ext[at[:, j]]).sum(0) for j in range(W)], 1)
    return fwd, {"dx": dext[old:].to(dt).reshape(s["x"].shape), "dw": dw, "dbias": d.sum(0) if s["bias"] is not None else None,
                 "dstate": dext[:old].to(dt).reshape(n, W - 1, -1) if s["state"] is not None else None}


def _conv_step_plain(s):
    c, dt = s["case"], _dtype(s["case"])
    win = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (win.float() * s["w"].T).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    return (pre * _sigmoid(pre) if c["act"] else pre).to(dt), win[:, 1:].contiguous()


def _linear_scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is zero where a sequence starts."""
    shift = 1
    while shift < longest:
        b = torch.cat([b[:shift], b[shift:] + a[shift:] * b[:-shift]])
        a = torch.cat([a[:shift], a[shift:] * a[:-shift]])
        shift *= 2
    return b


def _scan_plain(s):
    c, dtype = s["case"], _dtype(s["case"])
    D, N, G = c["D"], c["N"], c["G"]
    Dg = D // G
    lead = s["x"].shape
    u, raw = (s[k].reshape(-1, G, Dg).float() for k in ("x", "dt"))
    Bm, Cm = (s[k].reshape(-1, G, 1, N).float() for k in ("Bm", "Cm"))
    A, skip, n = s["A"].view(G, Dg, N), s["D_skip"].view(G, Dg), len(s["lens"])
    raw = raw + s["dt_bias"].view(G, Dg)
    dt = _softplus(raw)
    a = torch.exp(dt[..., None] * A)
    b = (dt * u)[..., None] * Bm
    some = [i for i in range(n) if s["lens"][i]]
    h0 = s["h"].view(n, G, Dg, N) if s["h"] is not None else a.new_zeros(n, G, Dg, N)
    starts, ends = s["first"][some], s["end"][some] - 1
    a0 = a.clone()
    b[starts] += a[starts] * h0[some]
    a0[starts] = 0
    h = _linear_scan(a0, b, max(s["lens"]))
    del a0, b
    y = (h * Cm).sum(-1) + skip * u
    h_T = h0.clone()
    h_T[some] = h[ends]
    if s["z"] is not None:
        z = s["z"].reshape(-1, G, Dg).float()
        sz = _sigmoid(z)
        out = y * z * sz
    else:
        out = y
    out = out.to(dtype).reshape(lead), h_T.view(n, D, N)
    if not c["train"]:
        return out
    d = s["dy"].reshape(-1, G, Dg).float()
    dz = None
    if s["z"] is not None:
        dz = (d * y * sz * (1 + z * (1 - sz))).to(dtype).reshape(lead)
        d = d * z * sz
    b = d[..., None] * Cm
    b[ends] += s["dh_T"].view(n, G, Dg, N)[some]
    ar = torch.cat([a[1:], torch.zeros_like(a[:1])])
    ar[ends] = 0
    g = _linear_scan(ar.flip(0), b.flip(0), max(s["lens"])).flip(0)
    del ar, b
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[starts] = h0[some]
    dC = (d[..., None] * h).sum(2)
    dB = (g * (dt * u)[..., None]).sum(2)
    gB = (g * Bm).sum(-1)
    ag = a * g
    dh0 = s["dh_T"].view(n, G, Dg, N).clone()
    dh0[some] = ag[starts]
    w = ag * before
    ddt = ((w * A).sum(-1) + gB * u) * _sigmoid(raw)
    return out + ({"du": (dt * gB + skip * d).to(dtype).reshape(lead), "ddt": ddt.to(dtype).reshape(lead),
                   "dA": (w * dt[..., None]).sum(0).view(D, N), "dB": dB.to(dtype).reshape(s["Bm"].shape), "dC": dC.to(dtype).reshape(s["Cm"].shape),
                   "dD_skip": (d * u).sum(0).view(D), "dz": dz, "ddt_bias": ddt.sum(0).view(D), "dh0": dh0.view(n, D, N) if c["init"] else None},)


def _scan_step_plain(s):
    c, dtype = s["case"], _dtype(s["case"])
    n, D, N, G = c["seqs"], c["D"], c["N"], c["G"]
    u = s["x"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    Bm, Cm = (s[k].float().view(n, G, 1, N).expand(n, G, D // G, N).reshape(n, D, N) for k in ("Bm", "Cm"))
    h = torch.exp(dt[..., None] * s["A"]) * s["h"] + (dt * u)[..., None] * Bm
    y = (h * Cm).sum(-1) + s["D_skip"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(dtype), h


PLAIN = {"norm": _norm_plain, "conv": _conv_plain, "conv_step": _conv_step_plain, "scan": _scan_plain, "scan_step": _scan_step_plain}


def run(s):
    return _run_own(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    D, op = case["D"], case["op"]
    if op == "norm":
        x = case["rows"] * D
        gate, pre = case["gate"] != "none", case["pre"]
        if not case["train"]:
            return {"bytes": e * x * (3 + gate + pre), "flops": 12 * x}
        # forward: y, x, gate in, x_out, h out; gradient: dx_out, dh in, dy, dx, dgate out
        return {"bytes": e * x * ((3 + gate + pre) + (3 + pre + gate)), "flops": 40 * x}
    n, L = case["seqs"], case["seqs"] if op.endswith("_step") else case["tokens"]
    x = L * D
    if op == "conv_step":
        return {"bytes": e * x * 2 * case["W"], "flops": 2 * x * case["W"]}
    if op == "conv":
        states = e * n * D * (case["W"] - 1)
        if not case["train"]:
            return {"bytes": 2 * e * x + states * (1 + case["init"]), "flops": (2 * case["W"] + 4) * x}
        return {"bytes": 4 * e * x + states * (1 + 2 * case["init"]), "flops": (8 * case["W"] + 16) * x}
    N, G, z = case["N"], case["G"], case["z"]
    h = 4 * n * D * N
    bc = 2 * e * L * G * N
    if op == "scan_step":
        return {"bytes": e * x * (3 + z) + bc + 2 * h, "flops": 7 * x * N}
    if not case["train"]:
        return {"bytes": e * x * (3 + z) + bc + h * (1 + case["init"]), "flops": 7 * x * N}
    # inputs u, dt, z, B, C and the adjoints in; y, the gradients and the states out
    return {"bytes": e * x * ((2 + z) + 2 + (2 + z)) + 2 * bc + h * (2 + 2 * case["init"]), "flops": 28 * x * N}


# ------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "conv": _conv_exact, "conv_step": _conv_step_exact, "scan": _scan_exact, "scan_step": _scan_step_exact}[case["op"]](s)


def _leaf(t, grad):
    return None if t is None else t.detach().double().clone().requires_grad_(grad)


def _grad(t):
    return None if t is None else t.grad


def _norm_exact(s):
    c = s["case"]
    train = c["train"]
    y, x, gate, w1, w2, scale = (_leaf(s[k], train) for k in ("y", "x", "gate", "w_post", "w_pre", "scale"))
    b = y if w1 is None else y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * w1
    if gate is not None:
        b = b * (gate.sigmoid() if c["gate"] == "sigmoid" else torch.nn.functional.silu(gate))
    X = x + (b if scale is None else b * scale)
    h = None if w2 is None else X / (X.square().mean(-1, keepdim=True) + EPS).sqrt() * w2
    if not train:
        return X, h
    ((X * s["dx_out"].double()).sum() + (0 if h is None else (h * s["dh"].double()).sum())).backward()
    return X.detach(), None if h is None else h.detach(), {"dy": y.grad, "dx": x.grad, "dgate": _grad(gate), "dw_post": _grad(w1), "dw_pre": _grad(w2), "dscale": _grad(scale)}


def _conv_exact(s):
    c = s["case"]
    train, W, D = c["train"], c["W"], c["D"]
    x, w, bias, state = (_leaf(s[k], train) for k in ("x", "w", "bias", "state"))
    rows, out, last, at = x.reshape(-1, D), [], [], 0
    for i, n in enumerate(s["lens"]):
        head = x.new_zeros(W - 1, D) if state is None else state[i]
        seq = torch.cat([head, rows[at:at + n]])
        at += n
        if n:
            out.append((seq.unfold(0, W, 1) * w).sum(-1))
        last.append(seq[n:])
    pre = torch.cat(out) + (0 if bias is None else bias)
    y = (torch.nn.functional.silu(pre) if c["act"] else pre).reshape(x.shape)
    fwd = y.detach(), torch.stack(last).detach()
    if not train:
        return fwd
    (y * s["dy"].double()).sum().backward()
    return fwd, {"dx": x.grad, "dw": w.grad, "dbias": _grad(bias), "dstate": _grad(state)}


def _conv_step_exact(s):
    x, w, state = (s[k].double() for k in ("x", "w", "state"))
    pre = x * w[:, -1] + sum(state[:, j] * w[:, j] for j in range(state.shape[1]))
    if s["bias"] is not None:
        pre = pre + s["bias"].double()
    return torch.nn.functional.silu(pre) if s["case"]["act"] else pre, torch.cat([state[:, 1:], x[:, None]], 1)


def _padded(t, lens):
    """[longest, sequences, ...] of a packed or batched [.., ...] tensor, zeros behind each sequence's end."""
    out = t.new_zeros((max(lens), len(lens)) + t.shape[1:])
    at = 0
    for i, n in enumerate(lens):
        out[:n, i] = t[at:at + n]
        at += n
    return out


def _unpadded(t, lens):
    return torch.cat([t[:n, i] for i, n in enumerate(lens)])


def _scan_exact(s):
    c, lens = s["case"], s["lens"]
    train, D, N, G, T, n = c["train"], c["D"], c["N"], c["G"], max(s["lens"]), len(s["lens"])
    if train and (T > 6000 or T * n * D * N > 1.2e9):
        return None
    lead = s["x"].shape
    leaf = {k: _leaf(_padded(s[k].reshape((-1,) + s[k].shape[2:]).double(), lens) if k in ("x", "dt", "Bm", "Cm", "z") and s[k] is not None else s[k], train)
            for k in ("x", "dt", "Bm", "Cm", "z", "A", "D_skip", "dt_bias", "h")}
    live = _padded(torch.ones(sum(lens), device=DEV, dtype=torch.float64), lens)[..., None]
    size = torch.nn.functional.softplus(leaf["dt"] + leaf["dt_bias"], threshold=40.0) * live
    h = leaf["h"] if leaf["h"] is not None else torch.zeros(n, D, N, device=DEV, dtype=torch.float64)
    rows = []
    for t in range(T):
        Bt, Ct = (leaf[k][t].repeat_interleave(D // G, dim=1) for k in ("Bm", "Cm"))
        h = h * torch.exp(size[t, ..., None] * leaf["A"]) + (size[t] * leaf["x"][t])[..., None] * Bt
        rows.append(torch.einsum("sdn,sdn->sd", h, Ct))
    y = torch.stack(rows) + leaf["D_skip"] * leaf["x"]
    if leaf["z"] is not None:
        y = y * torch.nn.functional.silu(leaf["z"])
    out = _unpadded(y.detach(), lens).reshape(lead), h.detach()
    if not train:
        return out
    ((y * _padded(s["dy"].reshape(-1, D).double(), lens)).sum() + (h * s["dh_T"].double()).sum()).backward()

    def rows_of(k):
        return None if leaf[k] is None else _unpadded(leaf[k].grad, lens).reshape(s[k].shape)

    return out + ({"du": rows_of("x"), "ddt": rows_of("dt"), "dA": leaf["A"].grad, "dB": rows_of("Bm"), "dC": rows_of("Cm"), "dD_skip": leaf["D_skip"].grad,
                   "dz": rows_of("z"), "ddt_bias": leaf["dt_bias"].grad, "dh0": _grad(leaf["h"])},)


def _scan_step_exact(s):
    c = s["case"]
    u, dt, A, h = (s[k].double() for k in ("x", "dt", "A", "h"))
    Bt, Ct = (s[k].double().repeat_interleave(c["D"] // c["G"], dim=1) for k in ("Bm", "Cm"))
    size = torch.nn.functional.softplus(dt + s["dt_bias"].double(), threshold=40.0)
    h = h * torch.exp(size[..., None] * A) + (size * u)[..., None] * Bt
    y = torch.einsum("sdn,sdn->sd", h, Ct) + s["D_skip"].double() * u
    return (y if s["z"] is None else y * torch.nn.functional.silu(s["z"].double())), h
