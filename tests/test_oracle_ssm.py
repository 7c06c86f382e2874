"""The fp64 reference of the state-space layer's operators, pinned on the CPU:
its forward against closed forms and an independent evaluation, its gradients
against central differences of its own forward."""
import numpy as np
import pytest

from oracle import ssm


def _numeric(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + h
        hi = f()
        x[i] = keep - h
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * h)
    return g


# central differences of a smooth function: h^2 f''' / 6 + 2^-53 f / h, with
# h = 1e-5 and values of order 10: about 1e-9 each
DIFF = dict(rtol=1e-6, atol=1e-7)


def _scan_case(seed, z=True, softplus=True, G=2):
    r = np.random.default_rng(seed)
    cu, D, N = [0, 3, 3, 5, 6], 4, 3
    L, S = cu[-1], len(cu) - 1
    sign = (lambda v: v) if softplus else np.abs       # steps of the plain form are positive
    return dict(u=r.normal(size=(L, D)), dt=sign(r.normal(size=(L, D)) * 0.5), A=-np.exp(r.normal(size=(D, N))),
                Bm=r.normal(size=(L, G, N)), Cm=r.normal(size=(L, G, N)), D_skip=r.normal(size=D),
                z=r.normal(size=(L, D)) if z else None, dt_bias=sign(r.normal(size=D)),
                h0=r.normal(size=(S, D, N)), cu=cu, use_softplus=softplus)


@pytest.mark.parametrize("z,softplus,G", [(True, True, 2), (False, True, 1), (True, False, 4)])
def test_scan_gradient_against_differences(z, softplus, G):
    c = _scan_case(1, z, softplus, G)
    r = np.random.default_rng(2)
    dy, dh = r.normal(size=c["u"].shape), r.normal(size=c["h0"].shape)

    def loss():
        y, hT, _ = ssm.scan(**c)
        return (y * dy).sum() + (hT * dh).sum()

    g = ssm.scan(**c, dy=dy, dh_T=dh)[3]
    names = dict(u="du", dt="ddt", A="dA", Bm="dB", Cm="dC", D_skip="dD_skip", dt_bias="ddt_bias", h0="dh0")
    if z:
        names["z"] = "dz"
    for k, d in names.items():
        np.testing.assert_allclose(g[d], _numeric(loss, c[k]), err_msg=d, **DIFF)


def test_scan_closed_form():
    # constant decay and input: h_T = b (1 - a^T) / (1 - a), y = C h + D u
    T, a, d = 7, 0.6, 0.5
    A = np.array([[np.log(a) / d]])
    y, hT, _ = ssm.scan(np.full((T, 1), 2.0), np.full((T, 1), d), A, np.full((T, 1, 1), 3.0),
                        np.full((T, 1, 1), 0.25), D_skip=np.array([10.0]), cu=[0, T], use_softplus=False)
    want = d * 2.0 * 3.0 * (1 - a ** np.arange(1, T + 1)) / (1 - a)
    np.testing.assert_allclose(hT[0, 0, 0], want[-1], rtol=1e-14)
    np.testing.assert_allclose(y[:, 0], 0.25 * want + 20.0, rtol=1e-14)


def test_scan_continues_from_a_state():
    c = _scan_case(3)
    c.update(cu=[0, 6], h0=c["h0"][:1])
    y, hT, _ = ssm.scan(**c)
    cut = lambda a, b: {k: v[a:b] if k in ("u", "dt", "Bm", "Cm", "z") else v for k, v in c.items()}
    y1, h1, _ = ssm.scan(**{**cut(0, 2), "cu": [0, 2]})
    y2, h2, _ = ssm.scan(**{**cut(2, 6), "cu": [0, 4], "h0": h1})
    np.testing.assert_allclose(np.concatenate([y1, y2]), y, rtol=1e-13)
    np.testing.assert_allclose(h2, hT, rtol=1e-13)


@pytest.mark.parametrize("W,silu,bias", [(2, True, True), (3, False, False), (4, True, False)])
def test_conv_gradient_against_differences(W, silu, bias):
    r = np.random.default_rng(W)
    cu, D = [0, 0, 5, 6, 6, 8], 3
    x, w = r.normal(size=(8, D)), r.normal(size=(D, W))
    b, st = r.normal(size=D) if bias else None, r.normal(size=(5, W - 1, D))
    dy, ds = r.normal(size=x.shape), r.normal(size=st.shape)

    def loss():
        y, last = ssm.conv(x, w, b, st, cu, silu)
        return (y * dy).sum() + (last * ds).sum()

    g = ssm.conv(x, w, b, st, cu, silu, dy=dy, dstate_T=ds)[2]
    for arr, d in ((x, "dx"), (w, "dw"), (st, "dstate")) + (((b, "dbias"),) if bias else ()):
        np.testing.assert_allclose(g[d], _numeric(loss, arr), err_msg=d, **DIFF)


def test_conv_against_numpy_convolve():
    r = np.random.default_rng(5)
    x, w = r.normal(size=(9, 2)), r.normal(size=(2, 4))
    y, last = ssm.conv(x, w, None, None, [0, 9], silu=False)
    for c in range(2):
        np.testing.assert_allclose(y[:, c], np.convolve(x[:, c], w[c, ::-1])[:9], rtol=1e-12, atol=1e-14)
    np.testing.assert_array_equal(last[0], x[-3:])


@pytest.mark.parametrize("post,pre,gate,scale", [(True, True, "sigmoid", True), (True, True, "silu", False),
                                                 (False, True, None, True), (True, False, None, False),
                                                 (False, False, "silu", True)])
def test_norm_gradient_against_differences(post, pre, gate, scale):
    r = np.random.default_rng(7)
    R, D = 3, 5
    y, x = r.normal(size=(R, D)), r.normal(size=(R, D))
    w1, w2 = r.normal(size=D) if post else None, r.normal(size=D) if pre else None
    g = r.normal(size=(R, D)) if gate else None
    sc = r.normal(size=D) if scale else None
    kw = dict(w_post=w1, w_pre=w2, gate=g, gate_act=gate or "sigmoid", scale=sc, eps=1e-3)
    dX, dh = r.normal(size=(R, D)), r.normal(size=(R, D)) if pre else None

    def loss():
        X, h = ssm.norm(y, x, **kw)
        return (X * dX).sum() + ((h * dh).sum() if pre else 0.0)

    got = ssm.norm(y, x, dx_out=dX, dh=dh, **kw)[2]
    for arr, d in ((y, "dy"), (x, "dx"), (g, "dgate"), (w1, "dw_post"), (w2, "dw_pre"), (sc, "dscale")):
        if arr is not None:
            np.testing.assert_allclose(got[d], _numeric(loss, arr), err_msg=d, **DIFF)
