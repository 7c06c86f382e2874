"""fp64 reference of linear attention with a decay for each head and of the
group norm with an activation (test infrastructure), token by token, each with
its gradient written out from its formula.

``magnitude=True`` evaluates the same formulas with every product and sum taken
over absolute values: what the rounding errors of an evaluation of the operator
are proportional to.
"""
import numpy as np


def linear_attn(q, k, v, log_decay, scale, S0=None, cu=None, do=None, dS_T=None, magnitude=False, exponent_error=0.0):
    """q [L, H, dk], k [L, Hkv, dk], v [L, Hkv, dv], S0 [S, H, dk, dv], cu [S+1].

    Returns (o [L, H, dv], S_T); with do a third, dict(dq, dk, dv, dS0).  With
    ``exponent_error`` e every decay a token is larger by the factor 1 + e |log
    decay|: twice evaluated, the difference bounds what an error e of the
    exponents makes."""
    ab = np.abs if magnitude else (lambda t: t)
    q, k, v, scale = ab(q), ab(k), ab(v), abs(scale) if magnitude else scale
    L, H, dk = q.shape
    Hkv, dv = v.shape[1:]
    S, shared = len(cu) - 1, H // Hkv
    lam = np.exp(np.maximum(log_decay, -1e30))
    if exponent_error:
        lam = lam * (1.0 + exponent_error * np.abs(np.maximum(log_decay, -700.0)))
    lam = lam[:, None, None]
    kk, vv = np.repeat(k, shared, axis=1), np.repeat(v, shared, axis=1)
    o, S_T, states = np.zeros((L, H, dv)), np.zeros((S, H, dk, dv)), None
    if do is not None:
        states = np.zeros((L, H, dk, dv))
    for s in range(S):
        Z = ab(S0[s]).copy() if S0 is not None else np.zeros((H, dk, dv))
        for t in range(cu[s], cu[s + 1]):
            Z = lam * Z + kk[t][:, :, None] * vv[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], Z)
            if states is not None:
                states[t] = Z
        S_T[s] = Z
    if do is None:
        return o, S_T
    do = ab(do)
    g = dict(dq=np.zeros((L, H, dk)), dk=np.zeros((L, H, dk)), dv=np.zeros((L, H, dv)), dS0=np.zeros((S, H, dk, dv)))
    for s in range(S):
        R = ab(dS_T[s]).copy() if dS_T is not None else np.zeros((H, dk, dv))
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            R = R + scale * q[t][:, :, None] * do[t][:, None, :]
            g["dq"][t] = scale * np.einsum("hkv,hv->hk", states[t], do[t])
            g["dk"][t] = np.einsum("hkv,hv->hk", R, vv[t])
            g["dv"][t] = np.einsum("hkv,hk->hv", R, kk[t])
            R = lam * R
        g["dS0"][s] = R
    g["dk"] = g["dk"].reshape(L, Hkv, shared, dk).sum(2)
    g["dv"] = g["dv"].reshape(L, Hkv, shared, dv).sum(2)
    return o, S_T, g


def _sig(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def act(x, name):
    """An activation, its derivative and a bound of its second one."""
    if name in (None, "none"):
        return x, np.ones_like(x), 0.0
    s = _sig(x)
    if name == "sigmoid":
        return s, s * (1 - s), 0.1
    return x * s, s * (1 + x * (1 - s)), 0.5


def group_norm(x, groups, weight=None, bias=None, gate=None, activation=None, cu=None, center=True, eps=1e-5, dy=None):
    """x [L, D]; groups of each token (cu None) or of each sequence.

    Returns (y, stats [n, G, 2]); with dy a third, dict(dx, dgate, dw, dbias)."""
    L, D = x.shape
    G = groups
    w = weight if weight is not None else np.ones(D)
    b = bias if bias is not None else np.zeros(D)
    runs = [(t, t + 1) for t in range(L)] if cu is None else list(zip(cu[:-1], cu[1:]))
    stats, n, dn_of = np.zeros((len(runs), G, 2)), np.zeros((L, D)), {}
    for i, (a, e) in enumerate(runs):
        if a == e:
            continue
        t = x[a:e].reshape(e - a, G, -1)
        mean = t.mean((0, 2)) if center else np.zeros(G)
        r = 1.0 / np.sqrt(((t - mean[:, None]) ** 2).mean((0, 2)) + eps)
        n[a:e] = ((t - mean[:, None]) * r[:, None]).reshape(e - a, D)
        stats[i, :, 0], stats[i, :, 1] = mean, r
    u = n * w + b
    if gate is None:
        y, du_y, _ = act(u, activation)
    else:
        ga, dga, _ = act(gate, activation)
        y = u * ga
    if dy is None:
        return y, stats
    du = dy * (du_y if gate is None else ga)
    dn = du * w
    dx = np.zeros((L, D))
    for i, (a, e) in enumerate(runs):
        if a == e:
            continue
        d, m = dn[a:e].reshape(e - a, G, -1), n[a:e].reshape(e - a, G, -1)
        out = d - m * (d * m).mean((0, 2))[:, None]
        if center:
            out = out - d.mean((0, 2))[:, None]
        dx[a:e] = (out * stats[i, :, 1][:, None]).reshape(e - a, D)
    return y, stats, dict(dx=dx, dgate=None if gate is None else dy * u * dga, dw=(du * n).sum(0), dbias=du.sum(0))
