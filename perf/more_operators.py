"""What is measured of linear attention with a decay for each head, and of the
group norm with an activation that follows it.

Every case names one operator and one way of using it: over whole prompts, in
a training step (forward and gradient), or for one token per sequence.  Where
``own`` is false ``run`` computes the operator from elementary torch
operations in 32 bits; where it is true it makes the library's calls.

Sizes are those of this repository's workloads (16 heads of 128 over 32768
packed tokens in 21 sequences and over 1 x 16384 tokens, 8 heads of 128 over
8 x 2048 tokens, 2 heads of 64 over 256 tokens, 256 decoding sequences, model
width 2048) and generic ones: shared key and value heads, odd widths.
"""
import math
import random

import torch

own = False
DEV = "cuda"
EPS = 1e-5
C = 128                # tokens of a chunk in the plain form


# ------------------------------------------------------------------ cases

def listed():
    bf, fp = "bf16", "fp32"
    return [
        # the whole prompts of a packed batch, as a server or an evaluation runs them
        attn("attn_prompts_packed", seqs=21, tokens=32768, packed=True, H=16, Hkv=16, dk=128, dv=128, dtype=bf, init=False),
        # one long document continued from a stored state: few heads' worth of parallel work
        attn("attn_long_prompt", seqs=1, tokens=16384, H=16, Hkv=16, dk=128, dv=128, dtype=bf, init=True),
        # a training step of the layer at 8 x 2048 tokens
        attn("attn_train_step", seqs=8, tokens=16384, H=8, Hkv=8, dk=128, dv=128, dtype=bf, init=False, train=True),
        # ragged training in fp32 with odd head widths, key and value heads shared by two query heads
        attn("attn_train_ragged_shared", seqs=5, tokens=1531, packed=True, H=6, Hkv=3, dk=40, dv=72, dtype=fp, init=True, train=True),
        # a short prompt of a small model in fp32: latency
        attn("attn_short_prompt", seqs=1, tokens=256, H=2, Hkv=2, dk=64, dv=64, dtype=fp, init=False),
        # one token for each of 256 decoding sequences, and for a few sequences of a small model (latency)
        dict(name="attn_decode", op="attn_step", seqs=256, H=16, Hkv=16, dk=128, dv=128, dtype=bf),
        dict(name="attn_decode_few", op="attn_step", seqs=4, H=8, Hkv=2, dk=64, dv=64, dtype=bf),
        # the norm of each head's output under a SiLU gate: prompts, a training step, decoding rows of odd groups
        norm("norm_heads_prompts", seqs=1, tokens=32768, D=2048, G=16, dtype=bf, gate=True, act="silu"),
        norm("norm_heads_train_step", seqs=8, tokens=16384, D=2048, G=16, dtype=bf, gate=True, act="silu", train=True),
        norm("norm_decode_odd_groups", seqs=1, tokens=64, D=1001, G=7, dtype=fp, gate=True, act="silu", center=False),
        # a non-causal mixer's norm over whole sequences, SiLU behind it, and its training in ragged fp32
        norm("norm_sequences", seqs=8, tokens=16384, D=2048, G=32, dtype=bf, gate=False, act="silu", over="sequence"),
        norm("norm_sequences_train_ragged", seqs=5, tokens=1531, packed=True, D=330, G=6, dtype=fp, gate=False, act="silu", over="sequence", train=True),
    ]


def attn(name, *, seqs, tokens, H, Hkv, dk, dv, dtype, init, packed=False, train=False):
    return dict(name=name, op="attn", seqs=seqs, tokens=tokens, packed=packed, H=H, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, init=init, train=train)


def norm(name, *, seqs, tokens, D, G, dtype, gate, act, packed=False, over="token", center=True, train=False):
    return dict(name=name, op="norm", seqs=seqs, tokens=tokens, packed=packed, D=D, G=G, dtype=dtype, gate=gate, act=act, over=over, center=center, train=train)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn_step", "norm", "norm"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op.startswith("attn"):
        c["Hkv"] = rng.choice([1, 2, 3, 4, 8, 16])
        c["H"] = c["Hkv"] * rng.choice([1, 1, 1, 2, 4])
        c["dk"], c["dv"] = (rng.choice([32, 64, 64, 96, 128, 128, 128, rng.randint(16, 128)]) for _ in range(2))
        if rng.random() < 0.5:
            c["dv"] = c["dk"]
    size = c["H"] * c["dk"] * c["dv"] if op != "norm" else 0
    if op == "attn_step":
        c["seqs"] = _log_int(rng, 1, max(1, min(1024, (1 << 26) // size)))
    elif op == "attn":
        c["train"], c["init"], c["packed"] = rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5
        most = max(1, min(32768, (1 << (30 if c["train"] else 32)) // size))
        c["seqs"] = _log_int(rng, 1, min(16, most))
        c["tokens"] = _log_int(rng, c["seqs"], most) if c["packed"] else c["seqs"] * _log_int(rng, 1, max(1, most // c["seqs"]))
    else:
        c["G"] = rng.choice([1, 2, 4, 7, 8, 16, 16, 32])
        c["D"] = c["G"] * _log_int(rng, 4, 4096 // c["G"])
        c.update(over=rng.choice(["token", "token", "sequence"]), center=rng.random() < 0.7, gate=rng.random() < 0.6, act=rng.choice(["silu", "silu", "sigmoid", "none"]),
                 train=rng.random() < 0.5, packed=rng.random() < 0.4)
        most = max(16, min(32768, (1 << 25) // c["D"]))
        c["seqs"] = rng.randint(1, 16)
        c["tokens"] = _log_int(rng, 16, most) if c["packed"] else c["seqs"] * _log_int(rng, 1, max(1, most // c["seqs"]))
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
    step = case["op"].endswith("_step")
    n = case["seqs"]
    if step:
        lead = (n,)
    else:
        lens = s["lens"] = _lengths(case, seed)
        lead = (1, case["tokens"]) if case["packed"] else (n, case["tokens"] // n)
        ends = torch.tensor(lens).cumsum(0)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).to(DEV) if case["packed"] else None
        s["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(lens)).to(DEV)
    if case["op"] == "norm":
        D = case["D"]
        s["x"] = randn(*lead, D, std=1.5, mean=0.3, dtype=dt)
        # the gate is one half of a wider projection
        s["gate"] = randn(*lead, 2 * D, dtype=dt)[..., D:] if case["gate"] else None
        s["weight"] = randn(D, std=0.2, mean=1.0)
        s["bias"] = randn(D, std=0.2) if case["center"] else None
        if case["train"]:
            s["dy"] = randn(*lead, D, dtype=dt)
        return s
    H, Hkv, dk, dv = (case[k] for k in ("H", "Hkv", "dk", "dv"))
    # q, k and v come out of one projection, side by side
    qkv = randn(*lead, H * dk + Hkv * (dk + dv), dtype=dt)
    q, k, v = qkv.split([H * dk, Hkv * dk, Hkv * dv], dim=-1)
    s["q"], s["k"], s["v"] = q.unflatten(-1, (H, dk)), k.unflatten(-1, (Hkv, dk)), v.unflatten(-1, (Hkv, dv))
    # time constants from two tokens to 256, geometrically over the heads
    s["log_decay"] = -torch.exp2(-8.0 * (torch.arange(H, device=DEV, dtype=torch.float32) + 1) / H) * torch.exp(randn(H, std=0.1))
    s["scale"] = dk ** -0.5
    s["S"] = randn(n, H, dk, dv) if step or case["init"] else None
    if step:
        s["S_out"] = torch.empty_like(s["S"])
        return s
    # the plain form's layout: chunks of a sequence, each token's chunk and place in it
    per = [-(-x // C) for x in lens]
    base = torch.tensor([0] + per).cumsum(0)[:-1]
    pos = torch.cat([torch.arange(x) for x in lens])
    s["chunk"], s["place"] = (base[s["seq"].cpu()] + pos // C).to(DEV), (pos % C).to(DEV)
    s["chunks"] = sum(per)
    s["chunk_seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(per)).to(DEV)
    s["chunk_pos"] = torch.cat([torch.arange(x) for x in per]).to(DEV) * C     # tokens of the sequence before each chunk
    s["len"] = torch.tensor(lens).to(DEV)
    if case["train"]:
        s["do"], s["dS_T"] = randn(*lead, H, dv, dtype=dt), randn(n, H, dk, dv)
    return s


# ------------------------------------------------------- the library's calls

def _run_own(s):
    import momentum_delta_rule_gb300 as mdn
    c = s["case"]
    if c["op"] == "norm":
        kw = dict(weight=s["weight"], bias=s["bias"], gate=s["gate"], activation=c["act"], over=c["over"], center=c["center"], cu_seqlens=s["cu"] if c["over"] == "sequence" else None, eps=EPS)
        if not c["train"]:
            return mdn.group_norm_fwd(s["x"], c["G"], **kw)
        y, stats = mdn.group_norm_fwd(s["x"], c["G"], return_stats=True, **kw)
        return y, mdn.group_norm_bwd(s["x"], c["G"], stats, s["dy"], **kw)
    args = (s["q"], s["k"], s["v"], s["log_decay"])
    if c["op"] == "attn_step":
        return mdn.linear_attn_step(*args, s["S"], scale=s["scale"], S_out=s["S_out"]), s["S_out"]
    kw = dict(scale=s["scale"], S0=s["S"], cu_seqlens=s["cu"])
    o, S_T = mdn.linear_attn_fwd(*args, **kw)
    if not c["train"]:
        return o, S_T
    return o, S_T, mdn.linear_attn_bwd(*args, s["do"], dS_T=s["dS_T"], need_dS0=c["init"], **kw)


# ------------------------------------------------------------ plain forms

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(x, act):
    """An activation and its derivative."""
    if act == "none":
        return x, torch.ones_like(x)
    sg = _sigmoid(x)
    return (sg, sg * (1 - sg)) if act == "sigmoid" else (x * sg, sg * (1 + x * (1 - sg)))


def _norm_plain(s):
    c, dt = s["case"], _dtype(s["case"])
    D, G = c["D"], c["G"]
    x = s["x"].reshape(-1, G, D // G).float()
    w = s["weight"].view(G, -1)
    if c["over"] == "token":
        def mean(t):
            return t.sum(2, keepdim=True) / (D // G)
    else:
        lens = torch.tensor(s["lens"], device=DEV)
        mine = (s["seq"] == torch.arange(c["seqs"], device=DEV)[:, None]).float()      # [n, tokens]

        def mean(t):
            return ((mine @ t.sum(2)) / (lens * (D // G)).clamp(min=1)[:, None])[s["seq"]][..., None]
    xc = x - mean(x) if c["center"] else x
    r = torch.rsqrt(mean(xc * xc) + EPS)
    n = xc * r
    u = n * w + (s["bias"].view(G, -1) if s["bias"] is not None else 0.0)
    if s["gate"] is not None:
        gate = s["gate"].reshape(-1, G, D // G).float()
        a, da = _act(gate, c["act"])
        y = u * a
    else:
        y, du = _act(u, c["act"])
    y = y.to(dt).reshape(s["x"].shape)
    if not c["train"]:
        return y
    dy = s["dy"].reshape(-1, G, D // G).float()
    du = dy * a if s["gate"] is not None else dy * du
    dn = du * w
    dx = dn - n * mean(dn * n)
    if c["center"]:
        dx = dx - mean(dn)
    return y, {"dx": (dx * r).to(dt).reshape(s["x"].shape), "dgate": (dy * u * da).to(dt).reshape(s["x"].shape) if s["gate"] is not None else None,
               "dw": (du * n).sum(0).view(D), "dbias": du.sum(0).view(D) if s["bias"] is not None else None}


def _in_chunks(s, t, H):
    """[chunks, H, C, width] in 32 bits of a [.., heads, width] tensor, zeros behind each sequence's end."""
    t = t.reshape(-1, *t.shape[-2:]).float()
    out = t.new_zeros(s["chunks"], C, *t.shape[1:])
    out[s["chunk"], s["place"]] = t
    return out.transpose(1, 2).repeat_interleave(H // t.shape[1], dim=1)


def _out_of_chunks(s, t, like, heads):
    """Back to the tokens' layout; query heads that share a key and value head are summed."""
    t = t.transpose(1, 2)[s["chunk"], s["place"]]
    return t.unflatten(1, (heads, -1)).sum(2).to(like.dtype).reshape(like.shape)


def _attn_plain(s):
    c = s["case"]
    H, Hkv, n = c["H"], c["Hkv"], c["seqs"]
    q, k, v = (_in_chunks(s, s[x], H) for x in ("q", "k", "v"))
    q = q * s["scale"]
    lam = s["log_decay"].double()
    seq, pos, left = s["chunk_seq"], s["chunk_pos"], s["len"][s["chunk_seq"]] - s["chunk_pos"]
    at = torch.arange(C, device=DEV)
    # the decay from token j to token i of a chunk, from before the chunk to i, and from j to the chunk's last token
    inside = torch.exp(lam[:, None, None] * (at[:, None] - at).clamp(min=0)).float() * (at[:, None] >= at)
    enter = torch.exp(lam[:, None] * (at + 1)).float()[..., None]
    end = (torch.minimum(left, torch.tensor(C, device=DEV))[:, None] - 1 - at).clamp(min=0)
    leave = torch.exp(lam[:, None] * end[:, None]).float()[..., None]
    # ... between chunks of one sequence, and between a sequence's ends and its chunks
    gap = pos[:, None] - pos - C
    across = torch.exp(lam[:, None, None] * gap.clamp(min=0)).float() * ((gap >= 0) & (seq[:, None] == seq))
    mine = seq == torch.arange(n, device=DEV)[:, None]                                         # [n, chunks]
    rest = (s["len"][:, None] - pos - C).clamp(min=0)
    behind = torch.exp(lam[:, None, None] * rest).float() * mine                                # a chunk's end -> the sequence's
    before = torch.exp(lam[:, None] * pos[:, None, None]).float().transpose(1, 2)[..., None]     # the sequence's start -> a chunk's
    whole = torch.exp(lam * s["len"][:, None]).float()[..., None, None]

    def mix(m, t):
        """Sums [H, a, b] x [b, H, x, y] -> [a, H, x, y] of states."""
        return (m @ t.transpose(0, 1).flatten(2)).unflatten(2, t.shape[2:]).transpose(0, 1)

    add = (k * leave).transpose(2, 3) @ v
    S = mix(across, add)
    S_T = mix(behind, add)
    if s["S"] is not None:
        S = S + before.reshape(-1, H, 1, 1) * s["S"][seq]
        S_T = S_T + whole * s["S"]
    A = (q @ k.transpose(2, 3)) * inside
    o = _out_of_chunks(s, A @ v + (q * enter) @ S, s["q"].new_empty(s["q"].shape[:-1] + (c["dv"],)), H)
    if not c["train"]:
        return o, S_T
    d = _in_chunks(s, s["do"], H)
    # the adjoint of the state behind each chunk, and of the initial one
    back = (q * enter).transpose(2, 3) @ d
    R = mix(across.transpose(1, 2), back) + behind.sum(1).T[..., None, None] * s["dS_T"][seq]
    first = torch.exp(lam[:, None, None] * pos).float() * mine
    dS0 = mix(first, back) + whole * s["dS_T"]
    B = (d @ v.transpose(2, 3)) * inside
    dq = (B @ k + (d * enter) @ S.transpose(2, 3)) * s["scale"]
    dk = B.transpose(2, 3) @ q + (v * leave) @ R.transpose(2, 3)
    dv = A.transpose(2, 3) @ d + (k * leave) @ R
    return o, S_T, {"dq": _out_of_chunks(s, dq, s["q"], H), "dk": _out_of_chunks(s, dk, s["k"], Hkv), "dv": _out_of_chunks(s, dv, s["v"], Hkv), "dS0": dS0 if c["init"] else None}


def _attn_step_plain(s):
    c = s["case"]
    shared = c["H"] // c["Hkv"]
    q, k, v = s["q"].float() * s["scale"], s["k"].float().repeat_interleave(shared, 1), s["v"].float().repeat_interleave(shared, 1)
    S = torch.exp(s["log_decay"])[:, None, None] * s["S"] + k[..., None] * v[..., None, :]
    return (q[..., None] * S).sum(2).to(_dtype(c)), S


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm_plain, "attn": _attn_plain, "attn_step": _attn_step_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        x, gate = case["tokens"] * case["D"], case["gate"]
        if not case["train"]:
            return {"bytes": e * x * (2 + gate), "flops": 12 * x}
        # forward: x, gate in, y out; gradient: dy in, dx, dgate out
        return {"bytes": e * x * (4 + 2 * gate), "flops": 36 * x}
    H, Hkv, dk, dv, n = (case[k] for k in ("H", "Hkv", "dk", "dv", "seqs"))
    L = n if case["op"] == "attn_step" else case["tokens"]
    qkv, o, state = L * (H * dk + Hkv * (dk + dv)), L * H * dv, 4 * n * H * dk * dv
    if case["op"] == "attn_step":
        return {"bytes": e * (qkv + o) + 2 * state, "flops": 5 * L * H * dk * dv}
    # the recurrence: a state's update and its product with q for each token
    flops = 5 * L * H * dk * dv
    if not case["train"]:
        return {"bytes": e * (qkv + o) + state * (1 + case["init"]), "flops": flops}
    # inputs and do in, o and the gradients out; states and their adjoints
    return {"bytes": e * (2 * qkv + 2 * o) + state * (2 + 2 * case["init"]), "flops": 4 * flops}


# ------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "attn": _attn_exact, "attn_step": _attn_step_exact}[case["op"]](s)


def _leaf(t, grad):
    return None if t is None else t.detach().double().clone().requires_grad_(grad)


def _norm_exact(s):
    c = s["case"]
    train, D, G = c["train"], c["D"], c["G"]
    x, gate, w, b = (_leaf(s[k], train) for k in ("x", "gate", "weight", "bias"))
    f = {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid, "none": lambda t: t}[c["act"]]
    rows, out, at = x.reshape(-1, D), [], 0
    for m in s["lens"] if c["over"] == "sequence" else [rows.shape[0]]:
        t = rows[at:at + m].unflatten(1, (G, -1))
        at += m
        if not m:
            continue
        dims = (0, 2) if c["over"] == "sequence" else (2,)
        if c["center"]:
            t = t - t.mean(dims, keepdim=True)
        out.append((t / (t.square().mean(dims, keepdim=True) + EPS).sqrt()).flatten(1))
    u = torch.cat(out).reshape(x.shape) * w
    if b is not None:
        u = u + b
    y = f(u) if gate is None else u * f(gate)
    if not train:
        return y.detach()
    (y * s["dy"].double()).sum().backward()
    return y.detach(), {"dx": x.grad, "dgate": None if gate is None else gate.grad, "dw": w.grad, "dbias": None if b is None else b.grad}


def _attn_exact(s):
    """Every sequence and head by itself, as one masked product over all pairs of tokens."""
    c, lens = s["case"], s["lens"]
    train, H, shared = c["train"], c["H"], c["H"] // c["Hkv"]
    if sum(m * m for m in lens) * H * (c["dk"] + c["dv"]) * (10 if train else 2) > 8e12:
        return None
    q, k, v, S = (_leaf(s[x], train) for x in ("q", "k", "v", "S"))
    flat = [t.reshape(-1, *t.shape[2:]) for t in (q, k, v)]
    o = torch.zeros(flat[0].shape[:2] + (c["dv"],), dtype=torch.float64, device=DEV)
    S_T = torch.zeros(c["seqs"], H, c["dk"], c["dv"], dtype=torch.float64, device=DEV)
    do = s["do"].double().reshape(o.shape) if train else None
    at = 0
    for i, m in enumerate(lens):
        t = torch.arange(m, device=DEV, dtype=torch.float64)
        for h in range(H):
            a = s["log_decay"][h].double()
            Q, K, V = flat[0][at:at + m, h] * s["scale"], flat[1][at:at + m, h // shared], flat[2][at:at + m, h // shared]
            out = (Q @ K.T * torch.exp(a * (t[:, None] - t)).tril()) @ V if m else Q @ K.T @ V
            last = (K * torch.exp(a * (m - 1 - t))[:, None]).T @ V
            if S is not None:
                out = out + torch.exp(a * (t + 1))[:, None] * (Q @ S[i, h])
                last = last + torch.exp(a * m) * S[i, h]
            if train:
                ((out * do[at:at + m, h]).sum() + (last * s["dS_T"][i, h].double()).sum()).backward(retain_graph=True)
            o[at:at + m, h], S_T[i, h] = out.detach(), last.detach()
        at += m
    o = o.reshape(s["q"].shape[:-1] + (c["dv"],))
    if not train:
        return o, S_T
    return o, S_T, {"dq": q.grad, "dk": k.grad, "dv": v.grad, "dS0": None if S is None else S.grad}


def _attn_step_exact(s):
    shared = s["case"]["H"] // s["case"]["Hkv"]
    q, k, v, S = (s[x].double() for x in ("q", "k", "v", "S"))
    S = S * torch.exp(s["log_decay"].double())[:, None, None] + torch.einsum("nhk,nhv->nhkv", k.repeat_interleave(shared, 1), v.repeat_interleave(shared, 1))
    return torch.einsum("nhk,nhkv->nhv", q * s["scale"], S), S
