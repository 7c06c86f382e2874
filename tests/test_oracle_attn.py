"""The fp64 references of linear attention and the group norm against other
forms of their definitions, and their gradients against differences."""
import numpy as np
import pytest

from oracle import attn


def _rng(seed=0):
    return np.random.default_rng(seed)


def _case(lens, H, Hkv, dk, dv, seed=0):
    r = _rng(seed)
    L, S = sum(lens), len(lens)
    cu = [0] + list(np.cumsum(lens))
    return dict(q=r.standard_normal((L, H, dk)), k=r.standard_normal((L, Hkv, dk)), v=r.standard_normal((L, Hkv, dv)),
                log_decay=-r.random(H), scale=0.3, S0=r.standard_normal((S, H, dk, dv)), cu=cu)


def test_linear_attention_is_a_masked_product():
    c = _case([5, 0, 9], 4, 2, 3, 6)
    o, S_T = attn.linear_attn(**c)
    for s in range(3):
        a, b = c["cu"][s], c["cu"][s + 1]
        n = b - a
        i = np.arange(n)
        for h in range(4):
            Q, K, V = c["q"][a:b, h], c["k"][a:b, h // 2], c["v"][a:b, h // 2]
            lam = np.exp(c["log_decay"][h])
            M = np.where(i[:, None] >= i, lam ** (i[:, None] - i), 0.0)
            want = 0.3 * ((Q @ K.T * M) @ V + lam ** (i + 1)[:, None] * (Q @ c["S0"][s, h]))
            np.testing.assert_allclose(o[a:b, h], want, rtol=1e-10, atol=1e-12)
            np.testing.assert_allclose(S_T[s, h], lam ** n * c["S0"][s, h] + (K * lam ** (n - 1 - i)[:, None]).T @ V,
                                       rtol=1e-10, atol=1e-12)


def test_a_decay_of_zero_forgets():
    c = _case([4], 2, 2, 3, 3)
    c["log_decay"] = np.array([-np.inf, 0.0])
    o, S_T = attn.linear_attn(**c)
    np.testing.assert_allclose(S_T[0, 0], np.outer(c["k"][3, 0], c["v"][3, 0]))
    np.testing.assert_allclose(o[:, 0], 0.3 * (c["q"][:, 0] * c["k"][:, 0]).sum(1, keepdims=True) * c["v"][:, 0])


def _differences(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        hi = f()
        x[i] = old - eps
        lo = f()
        x[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_linear_attention_gradient():
    c = _case([3, 0, 4], 4, 2, 3, 2, seed=1)
    r = _rng(2)
    do, dS_T = r.standard_normal((7, 4, 2)), r.standard_normal((3, 4, 3, 2))
    g = attn.linear_attn(**c, do=do, dS_T=dS_T)[2]

    def loss():
        o, S_T = attn.linear_attn(**c)
        return (o * do).sum() + (S_T * dS_T).sum()

    for name, x in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dS0", "S0")):
        np.testing.assert_allclose(g[name], _differences(loss, c[x]), rtol=1e-6, atol=1e-8, err_msg=name)


@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("cu,center", [(None, True), (None, False), ([0, 3, 3, 7], True), ([0, 3, 3, 7], False)])
def test_group_norm_gradient(activation, gated, cu, center):
    r = _rng(3)
    x, dy = r.standard_normal((7, 6)), r.standard_normal((7, 6))
    w, b = 1 + 0.3 * r.standard_normal(6), 0.2 * r.standard_normal(6)
    gate = r.standard_normal((7, 6)) if gated else None
    kw = dict(groups=2, weight=w, bias=b, gate=gate, activation=activation, cu=cu, center=center)
    y, stats, g = attn.group_norm(x, **kw, dy=dy)
    loss = lambda: (attn.group_norm(x, **kw)[0] * dy).sum()
    for name, t in (("dx", x), ("dw", w), ("dbias", b)) + ((("dgate", gate),) if gated else ()):
        np.testing.assert_allclose(g[name], _differences(loss, t), rtol=1e-5, atol=1e-8, err_msg=name)
    if activation is None and not gated and center:
        t = (y - b) / w
        for a, e in ([(i, i + 1) for i in range(7)] if cu is None else [(0, 3), (3, 7)]):
            z = t[a:e].reshape(e - a, 2, 3)
            np.testing.assert_allclose(z.mean((0, 2)), 0, atol=1e-12)
            # (below 1 by eps over the variance)
            assert (z.var((0, 2)) < 1).all()
