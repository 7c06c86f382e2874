"""fp64 reference of the state-space layer's operators (test infrastructure):
short causal convolution, selective scan and the norms around a block, each
with its gradient written out from its formula, token by token.

``magnitude=True`` evaluates the same formulas with every product and sum
taken over absolute values: what the rounding errors of an fp32 evaluation of
the operator are proportional to.
"""
import numpy as np


def _sig(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def _silu(x):
    return x * _sig(x)


def _dsilu(x):
    s = _sig(x)
    return s * (1.0 + x * (1.0 - s))


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


# -------------------------------------------------------------- convolution

def conv(x, w, bias, state, cu, silu=True, dy=None, dstate_T=None, magnitude=False):
    """x [L, D], w [D, W], bias [D] or None, state [S, W-1, D] or None, cu [S+1].

    Returns (y, state_T); with dy a third, dict(dx, dw, dbias, dstate)."""
    ab = np.abs if magnitude else (lambda v: v)
    L, D = x.shape
    W, S = w.shape[1], len(cu) - 1
    y, last = np.zeros((L, D)), np.zeros((S, W - 1, D))
    g = dict(dx=np.zeros((L, D)), dw=np.zeros((D, W)), dbias=np.zeros(D), dstate=np.zeros((S, W - 1, D)))
    for s in range(S):
        a, b = cu[s], cu[s + 1]
        head = state[s] if state is not None else np.zeros((W - 1, D))
        ext = np.concatenate([head, x[a:b]])
        last[s] = ext[b - a:]
        dext = np.zeros_like(ext)
        for t in range(b - a):
            win = ext[t:t + W]                               # [W, D]
            pre = (win * w.T).sum(0) + (bias if bias is not None else 0.0)
            size = (np.abs(win) * np.abs(w.T)).sum(0) + (np.abs(bias) if bias is not None else 0.0)
            if magnitude:
                y[a + t] = size
            else:
                y[a + t] = _silu(pre) if silu else pre
            if dy is not None:
                if magnitude:
                    # |act''| < 1: an error of pre moves act' by at most as much
                    e = np.abs(dy[a + t]) * (1.1 + (size if silu else 0.0))
                else:
                    e = dy[a + t] * (_dsilu(pre) if silu else 1.0)
                g["dbias"] += e
                g["dw"] += (e * ab(win)).T
                dext[t:t + W] += e * ab(w.T)
        if dstate_T is not None:
            dext[b - a:] += ab(dstate_T[s])
        g["dx"][a:b] = dext[W - 1:]
        g["dstate"][s] = dext[:W - 1]
    return (y, last) if dy is None else (y, last, g)


# --------------------------------------------------------------------- scan

def scan(u, dt, A, Bm, Cm, D_skip=None, z=None, dt_bias=None, h0=None, cu=None, use_softplus=True,
         dy=None, dh_T=None, magnitude=False):
    """u, dt, z [L, D]; A [D, N]; Bm, Cm [L, G, N]; h0 [S, D, N]; cu [S+1].

    Returns (y, h_T, states) with states [L, D, N] after every token; with dy a
    fourth, dict(du, ddt, dA, dB, dC, dD_skip, dz, ddt_bias, dh0)."""
    ab = np.abs if magnitude else (lambda v: v)
    L, D = u.shape
    G, N = Bm.shape[1:]
    S = len(cu) - 1
    rep = D // G
    raw = dt + (dt_bias if dt_bias is not None else 0.0)
    delta = softplus(raw) if use_softplus else raw
    dd = _sig(raw) if use_softplus else np.ones_like(raw)
    skip = D_skip if D_skip is not None else np.zeros(D)
    gate = _silu(z) if z is not None else np.ones_like(u)
    y, hs = np.zeros((L, D)), np.zeros((L, D, N))
    pre = np.zeros((L, D))
    h_T = np.zeros((S, D, N))
    dec = np.exp(delta[:, :, None] * A)
    dec[dec < 2.0 ** -126] = 0.0               # as the operator defines it
    for s in range(S):
        h = ab(h0[s]) if h0 is not None else np.zeros((D, N))
        for t in range(cu[s], cu[s + 1]):
            Bt, Ct = (np.repeat(ab(m[t]), rep, axis=0) for m in (Bm, Cm))
            h = dec[t] * h + (ab(delta[t]) * ab(u[t]))[:, None] * Bt
            hs[t] = h
            pre[t] = (h * Ct).sum(1) + ab(skip) * ab(u[t])
            y[t] = pre[t] * ab(gate[t])
        h_T[s] = h
    if dy is None:
        return y, h_T, hs
    g = dict(du=np.zeros((L, D)), ddt=np.zeros((L, D)), dA=np.zeros((D, N)), dB=np.zeros((L, G, N)),
             dC=np.zeros((L, G, N)), dD_skip=np.zeros(D), dz=np.zeros((L, D)), ddt_bias=np.zeros(D),
             dh0=np.zeros((S, D, N)))
    if z is not None:
        g["dz"] = ab(dy) * pre * (1.1 if magnitude else _dsilu(z))
    e = ab(dy) * ab(gate)
    for s in range(S):
        carry = ab(dh_T[s]) if dh_T is not None else np.zeros((D, N))
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            Bt, Ct = (np.repeat(ab(m[t]), rep, axis=0) for m in (Bm, Cm))
            if t > cu[s]:
                before = hs[t - 1]
            else:
                before = ab(h0[s]) if h0 is not None else np.zeros((D, N))
            gt = Ct * e[t][:, None] + carry
            du = ab(delta[t]) * ab(u[t])
            g["dB"][t] = (gt * du[:, None]).reshape(G, rep, N).sum(1)
            g["dC"][t] = (hs[t] * e[t][:, None]).reshape(G, rep, N).sum(1)
            s1 = (gt * Bt).sum(1)
            carry = dec[t] * gt
            w = carry * before
            g["du"][t] = ab(delta[t]) * s1 + ab(skip) * e[t]
            g["ddt"][t] = ((ab(A) * w).sum(1) + ab(u[t]) * s1) * dd[t]
            g["dA"] += ab(delta[t])[:, None] * w
            g["dD_skip"] += e[t] * ab(u[t])
            g["ddt_bias"] += g["ddt"][t]
        g["dh0"][s] = carry
    return y, h_T, hs, g


# -------------------------------------------------------------------- norms

def norm(y, x, w_post=None, w_pre=None, gate=None, gate_act="sigmoid", scale=None, eps=1e-6,
         dx_out=None, dh=None):
    """Rows [R, D].  Returns (x_out, h or None); with dx_out a third, dict(dy,
    dx, dgate, dw_post, dw_pre, dscale)."""
    D = y.shape[1]
    one = np.ones(D)
    r1 = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if w_post is not None else 1.0
    w1 = w_post if w_post is not None else one
    n = y * r1 * w1
    if gate is None:
        act, dact = 1.0, 0.0
    elif gate_act == "silu":
        act, dact = _silu(gate), _dsilu(gate)
    else:
        act = _sig(gate)
        dact = act * (1.0 - act)
    b = n * act
    sc = scale if scale is not None else one
    X = x + sc * b
    h = r2 = None
    if w_pre is not None:
        r2 = 1.0 / np.sqrt((X * X).mean(1, keepdims=True) + eps)
        h = X * r2 * w_pre
    if dx_out is None:
        return X, h
    g = {}
    dX = dx_out.copy()
    if w_pre is not None:
        g["dw_pre"] = (dh * X * r2).sum(0)
        dX += r2 * (w_pre * dh - X * r2 ** 2 * (dh * w_pre * X).mean(1, keepdims=True))
    g["dx"] = dX
    if scale is not None:
        g["dscale"] = (dX * b).sum(0)
    db = dX * sc
    if gate is not None:
        g["dgate"] = db * n * dact
    dn = db * act
    if w_post is not None:
        g["dw_post"] = (dn * y * r1).sum(0)
        dn = r1 * (w1 * dn - y * r1 ** 2 * (dn * w1 * y).mean(1, keepdims=True))
    g["dy"] = dn
    return X, h, g
