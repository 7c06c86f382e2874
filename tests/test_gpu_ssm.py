"""GPU parity of the state-space layer's operators against the fp64 reference
(``oracle/ssm.py``), element by element.

Tolerance of an output x with the magnitude m of its terms (the reference
formula over absolute values): half a step of its type, eps / 2 |x|, plus the
fp32 evaluation's own error, at most (K + c T) 2^-24 m.  A step of the
recurrence makes four roundings and one exp2 of relative error 2^-22 whose
argument carries two more: c = 16 covers it and the adjoint's the same way; K
= 64 covers the elementwise functions (softplus, sigmoid: a few 2^-22) and
the sums over lanes, channels and tokens outside the recurrence (at most one
rounding a term, T + D terms).
"""
import numpy as np
import pytest
import torch

from oracle import ssm

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _close(name, got, ref, mag, ulps, dtype=None):
    """|got - ref| <= eps/2 |ref| + ulps 2^-24 mag, with eps of got's type."""
    eps = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(g).all(), name
    # the rounding acts on the computed value: (1 + eps/2) covers its offset
    tol = eps * np.abs(ref) + (1 + eps) * ulps * 2.0 ** -24 * np.abs(mag) + 1e-37
    bad = np.abs(g - ref) > tol
    worst = float((np.abs(g - ref) / tol).max()) if ref.size else 0.0
    assert not bad.any(), "%s: %d of %d off, worst %.2f times the tolerance, at %s" % (
        name, bad.sum(), bad.size, worst, np.argwhere(bad)[:3].tolist())


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cu(lens):
    return [0] + list(np.cumsum(lens).tolist())


# -------------------------------------------------------------------- scan

def scan_case(dtype, lens, D, N, G=1, z=True, init=True, bias=True, skip=True, softplus=True, packed=True,
              strided=True, seed=0):
    g = _gen(seed)
    L, S = int(sum(lens)), len(lens)
    td = TD[dtype]
    rn = lambda *s: torch.randn(s, generator=g)
    lead = (1, L) if packed else (S, L // S)
    if strided:
        xz = rn(*lead, 2 * D + 8).to(td)
        u, zz = xz[..., :D], xz[..., D:2 * D]
        bc = rn(*lead, 2 * G * N + 8).to(td)
        Bm, Cm = (t.unflatten(-1, (G, N)) for t in (bc[..., :G * N], bc[..., G * N:2 * G * N]))
    else:
        u, zz = rn(*lead, D).to(td), rn(*lead, D).to(td)
        Bm, Cm = rn(*lead, G, N).to(td), rn(*lead, G, N).to(td)
    dt = (rn(*lead, D) * 0.7).to(td) if softplus else (rn(*lead, D).abs() * 0.2).to(td)
    return dict(u=u, dt=dt, Bm=Bm, Cm=Cm, z=zz if z else None,
                A=-torch.exp(rn(D, N)), D_skip=rn(D) if skip else None,
                dt_bias=(rn(D) - 2.0 if softplus else rn(D).abs() * 0.1) if bias else None,
                h0=rn(S, D, N) if init else None, softplus=softplus, lens=lens, packed=packed)


def _dev(c):
    """The case on the GPU, slices staying slices of one wider tensor."""
    out, moved = {}, {}
    for k, v in c.items():
        if isinstance(v, torch.Tensor):
            base = v._base if v._base is not None else v
            if id(base) not in moved:
                moved[id(base)] = base.cuda()
            v = torch.as_strided(moved[id(base)], v.shape, v.stride(), v.storage_offset())
        out[k] = v
    return out


def _scan_ref(c, **kw):
    L, D = int(sum(c["lens"])), c["u"].shape[-1]
    f = lambda t, *tail: None if t is None else _np(t).reshape(L, *tail)
    G, N = c["Bm"].shape[-2:]
    return ssm.scan(f(c["u"], D), f(c["dt"], D), _np(c["A"]), f(c["Bm"], G, N), f(c["Cm"], G, N),
                    _np(c["D_skip"]), f(c["z"], D), _np(c["dt_bias"]), _np(c["h0"]), _cu(c["lens"]),
                    c["softplus"], **kw)


def _scan_kw(d):
    cu = torch.tensor(_cu(d["lens"]), dtype=torch.int32).cuda() if d["packed"] else None
    return dict(D_skip=d["D_skip"], z=d["z"], dt_bias=d["dt_bias"], softplus=d["softplus"], cu_seqlens=cu)


def check_scan(c, train=False, dh=True, stream=None):
    import momentum_delta_rule_gb300 as mdn
    d = _dev(c)
    T = max(c["lens"]) if c["lens"] else 0
    D, N = d["A"].shape
    y, hT, hc = mdn.ssm_scan_fwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], h0=d["h0"],
                                 return_chunk_states=True, **_scan_kw(d))
    y2, hT2 = mdn.ssm_scan_fwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], h0=d["h0"], **_scan_kw(d))
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    assert torch.equal(y, y2) and torch.equal(hT, hT2)      # saving states changes no result
    kw = {}
    if train:
        g = _gen(99)
        dy = torch.randn(y.shape, generator=g).to(y.dtype)
        dhT = torch.randn(hT.shape, generator=g) if dh else None
        kw = dict(dy=_np(dy).reshape(-1, D), dh_T=_np(dhT))
    ref, mag = _scan_ref(c, **kw), _scan_ref(c, magnitude=True, **kw)
    ulps = 64 + 16 * T
    _close("y", y.reshape(-1, D), ref[0], mag[0], ulps)
    _close("h_T", hT, ref[1], mag[1], ulps)
    cu, slot = _cu(c["lens"]), 0
    for s, n in enumerate(c["lens"]):                       # the saved states
        for k in range((n + 31) // 32):
            if k:
                _close("h_chunks", hc[slot], ref[2][cu[s] + 32 * k - 1], mag[2][cu[s] + 32 * k - 1], ulps)
            else:
                want = torch.zeros(D, N) if c["h0"] is None else c["h0"][s]
                assert torch.equal(hc[slot].cpu(), want)
            slot += 1
    if not train:
        return
    grads = mdn.ssm_scan_bwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], hc, dy.cuda(),
                             dh_T=None if dhT is None else dhT.cuda(), need_dh0=True, **_scan_kw(d))
    again = mdn.ssm_scan_bwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], hc, dy.cuda(),
                             dh_T=None if dhT is None else dhT.cuda(), need_dh0=True, **_scan_kw(d))
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    L = sum(c["lens"])
    # sums over all tokens or all channels of a group: one rounding a term
    more = {"dA": L, "dD_skip": L, "ddt_bias": L, "dB": D, "dC": D}
    for k, v in grads.items():
        none = {"dD_skip": c["D_skip"], "dz": c["z"], "ddt_bias": c["dt_bias"]}.get(k, 1) is None
        assert (v is None) == none, k
        if v is None:
            continue
        assert torch.equal(v, again[k]), k                  # the same bits
        r, m = ref[3][k], mag[3][k]
        _close(k, v.reshape(r.shape), r, m, 2 * ulps + more.get(k, 0))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [1, 3, 4, 8, 16, 17, 32, 64, 100, 128])
def test_scan_state_sizes(dtype, N):
    check_scan(scan_case(dtype, [33, 7], D=24, N=N, seed=N), train=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D,G", [(1, 1), (7, 1), (20, 4), (66, 2), (130, 1), (129, 3), (264, 2)])
def test_scan_widths_and_groups(dtype, D, G):
    check_scan(scan_case(dtype, [5, 40, 1], D=D, N=16, G=G, seed=D), train=True)


@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [64, 65], [0, 1, 0, 0, 100, 0], [3] * 9, [200, 1, 130]])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_scan_lengths(dtype, lens):
    check_scan(scan_case(dtype, lens, D=32, N=16, seed=len(lens)), train=True)


@pytest.mark.parametrize("kw", [dict(z=False), dict(init=False), dict(bias=False), dict(skip=False),
                                dict(softplus=False), dict(z=False, init=False, bias=False, skip=False)])
@pytest.mark.parametrize("strided", [True, False])
def test_scan_options(kw, strided):
    check_scan(scan_case("fp32", [40, 9], D=36, N=16, G=2, strided=strided, **kw), train=True)
    check_scan(scan_case("bf16", [24, 24], D=36, N=12, packed=False, strided=strided, **kw), train=True, dh=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_scan_extreme_steps(dtype):
    # steps from where the state survives a whole sequence to where one token
    # wipes it out (decay underflows to 0), and softplus far out on both sides
    c = scan_case(dtype, [50, 20], D=32, N=16, seed=5)
    c["dt_bias"] = torch.linspace(-30.0, 60.0, 32)
    check_scan(c, train=True)
    c = scan_case(dtype, [50, 20], D=32, N=16, seed=6)
    c["A"][:, ::3] = 0.0                                   # a state that never decays
    check_scan(c, train=True)


def test_scan_state_without_decay_or_input_is_kept():
    # A = 0 or delta = 0 (exp(0) = 1), and B = 0: the state stays, bit for bit
    import momentum_delta_rule_gb300 as mdn
    c = _dev(scan_case("fp32", [501, 3], D=64, N=16, seed=14, softplus=False, bias=False))
    zero = torch.zeros_like(c["Bm"])
    for dt, A in ((c["dt"], torch.zeros_like(c["A"])), (torch.zeros_like(c["dt"]), c["A"])):
        _, hT = mdn.ssm_scan_fwd(c["u"], dt, A, zero, c["Cm"], h0=c["h0"], **_scan_kw(c))
        assert torch.equal(hT, c["h0"])
        h = c["h0"].clone()
        mdn.ssm_scan_step(c["u"][0, :2], dt[0, :2], A, zero[0, :2], c["Cm"][0, :2], h, softplus=False)
        assert torch.equal(h, c["h0"])


def test_scan_unaligned_rows():
    # rows and bases on no packet boundary
    c = scan_case("bf16", [37, 20], D=40, N=16, seed=8)
    wide = torch.randn(1, 57, 2 * 40 + 3, generator=_gen(9)).to(torch.bfloat16)
    c["u"], c["z"] = wide[..., 1:41], wide[..., 42:82]
    check_scan(c, train=True)


def test_scan_single_long_sequence_and_many_short():
    check_scan(scan_case("fp32", [1500], D=16, N=16, seed=11, packed=False), train=True)
    check_scan(scan_case("bf16", [3] * 300, D=16, N=8, seed=12), train=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,S,D,N,G", [(300, 2, 40, 16, 1), (97, 3, 34, 8, 2), (64, 1, 16, 16, 1), (65, 2, 9, 128, 1), (130, 40, 192, 32, 1)])
def test_scan_cut_sequences_of_equal_length(dtype, T, S, D, N, G):
    # few blocks: the forward and the gradient cut them into segments of their own
    check_scan(scan_case(dtype, [T] * S, D=D, N=N, G=G, packed=False, seed=T), train=True)


def test_scan_step_of_many_sequences():
    # more than the grid's second dimension holds
    import momentum_delta_rule_gb300 as mdn
    n = 65535 + 70
    g = _gen(40)
    u, dt, z = (torch.randn(n, 2, generator=g).cuda() for _ in range(3))
    A = -torch.rand(2, 1, generator=g).cuda()
    Bm, Cm, h = (torch.randn(*s, generator=g).cuda() for s in ((n, 1, 1), (n, 1, 1), (n, 2, 1)))
    out = torch.empty_like(h)
    y = mdn.ssm_scan_step(u, dt, A, Bm, Cm, h, z=z, h_out=out)
    rows = [0, 1, 65534, 65535, 65536, n - 1]
    part = torch.empty(len(rows), 2, 1, device="cuda")
    want = mdn.ssm_scan_step(u[rows], dt[rows], A, Bm[rows], Cm[rows], h[rows], z=z[rows], h_out=part)
    assert torch.equal(y[rows], want) and torch.equal(out[rows], part)


def test_scan_without_tokens():
    import momentum_delta_rule_gb300 as mdn
    c = _dev(scan_case("fp32", [0, 0], D=8, N=4, packed=False))
    y, hT, hc = mdn.ssm_scan_fwd(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], h0=c["h0"],
                                 return_chunk_states=True, **_scan_kw(c))
    assert y.shape == (2, 0, 8) and torch.equal(hT, c["h0"]) and hc.shape[0] == 0
    dh = torch.randn(2, 8, 4, device="cuda")
    g = mdn.ssm_scan_bwd(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], hc, y, dh_T=dh, need_dh0=True, **_scan_kw(c))
    assert torch.equal(g["dh0"], dh)
    for k in ("dA", "dD_skip", "ddt_bias"):
        assert not g[k].any()


def test_scan_final_state_in_place_and_given_buffers():
    import momentum_delta_rule_gb300 as mdn
    c = _dev(scan_case("bf16", [70, 5], D=64, N=16, seed=3))
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"])
    y, hT = mdn.ssm_scan_fwd(*args, h0=c["h0"], **_scan_kw(c))
    h = c["h0"].clone()
    out = torch.empty_like(y)
    y2, h2 = mdn.ssm_scan_fwd(*args, h0=h, h_T=h, y=out, **_scan_kw(c))
    assert h2 is h and y2 is out and torch.equal(h, hT) and torch.equal(out, y)


@pytest.mark.parametrize("lens,packed", [([1500, 1500], False), ([2001, 7], True), ([900], False)])
def test_scan_final_states_of_cut_sequences_in_place(lens, packed):
    import momentum_delta_rule_gb300 as mdn
    c = _dev(scan_case("bf16", lens, D=66, N=16, packed=packed, seed=4))
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"])
    y, hT = mdn.ssm_scan_fwd(*args, h0=c["h0"], **_scan_kw(c))
    h = c["h0"].clone()
    y2, h2 = mdn.ssm_scan_fwd(*args, h0=h, h_T=h, **_scan_kw(c))
    assert h2 is h and torch.equal(h, hT) and torch.equal(y2, y)


@pytest.mark.parametrize("cu", [[0, 40, 20, 60], [0, 20, 50], [5, 20, 60]])
def test_malformed_offsets_are_reported(cu):
    import momentum_delta_rule_gb300 as mdn
    n = len(cu) - 1
    c = _dev(scan_case("fp32", [60], D=8, N=4))
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h0 = torch.randn(n, 8, 4, device="cuda")
    y = torch.full((1, 60, 8), 7.0, device="cuda")
    kw = dict(D_skip=c["D_skip"], z=c["z"], dt_bias=c["dt_bias"], cu_seqlens=cud)
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"])
    _, hT, hc = mdn.ssm_scan_fwd(*args, h0=h0, y=y, return_chunk_states=True, **kw)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert torch.equal(hT, h0) and (y == 7.0).all()
    g = mdn.ssm_scan_bwd(*args, hc, torch.ones_like(y), dh_T=h0, need_dh0=True, **kw)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert torch.equal(g["dh0"], h0) and not g["dA"].any() and not g["ddt_bias"].any()
    x = torch.randn(1, 60, 8, device="cuda")
    w, st = torch.randn(8, 4, device="cuda"), torch.randn(n, 3, 8, device="cuda")
    y.fill_(7.0)
    _, last = mdn.short_conv_fwd(x, w, state=st, cu_seqlens=cud, y=y, output_final_state=True)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert torch.equal(last, st) and (y == 7.0).all()
    g = mdn.short_conv_bwd(x, w, y, state=st, cu_seqlens=cud, dstate_T=st)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert torch.equal(g["dstate"], st) and not g["dw"].any()
    assert mdn.device_status() == mdn.MDN_OK


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,D,N,G", [(1, 1, 1, 1), (3, 40, 16, 2), (5, 66, 5, 1), (2, 24, 128, 4), (64, 128, 16, 1), (3, 10, 33, 1)])
def test_scan_step(dtype, n, D, N, G):
    import momentum_delta_rule_gb300 as mdn
    c = scan_case(dtype, [1] * n, D=D, N=N, G=G, seed=n + D)
    d = _dev(c)
    kw = {k: d[k] for k in ("D_skip", "z", "dt_bias", "softplus")}
    two = lambda t: None if t is None else t[0]
    kw["z"] = two(kw["z"])
    args = [two(d["u"]), two(d["dt"]), d["A"], two(d["Bm"]), two(d["Cm"])]
    out = torch.empty_like(d["h0"])
    y = mdn.ssm_scan_step(*args, d["h0"], h_out=out, **kw)
    h = d["h0"].clone()
    y2 = mdn.ssm_scan_step(*args, h, **kw)
    torch.cuda.synchronize()
    ref, mag = _scan_ref(c), _scan_ref(c, magnitude=True)
    _close("y", y, ref[0], mag[0], 80 + N)
    _close("h", out, ref[1], mag[1], 80)
    assert torch.equal(h, out) and torch.equal(y, y2)


def test_scan_step_continues_a_prompt():
    import momentum_delta_rule_gb300 as mdn
    c = _dev(scan_case("fp32", [40, 40], D=32, N=16, packed=False, seed=21))
    kw = _scan_kw(c)
    kw.pop("cu_seqlens")
    args = lambda a, b: [c[k][:, a:b] for k in ("u", "dt")] + [c["A"]] + [c[k][:, a:b] for k in ("Bm", "Cm")]
    y, hT = mdn.ssm_scan_fwd(*[t.contiguous() for t in args(0, 40)], h0=c["h0"], **{**kw, "z": c["z"].contiguous()})
    _, h = mdn.ssm_scan_fwd(*[t.contiguous() for t in args(0, 33)], h0=c["h0"], **{**kw, "z": c["z"][:, :33].contiguous()})
    for t in range(33, 40):
        u, dt, A, Bm, Cm = args(t, t + 1)
        yt = mdn.ssm_scan_step(u[:, 0], dt[:, 0], A, Bm[:, 0], Cm[:, 0], h, **{**kw, "z": c["z"][:, t]})
        torch.testing.assert_close(yt, y[:, t], rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(h, hT, rtol=1e-5, atol=1e-5)


# ------------------------------------------------------------- convolution

def conv_case(dtype, lens, D, W, bias=True, init=True, packed=True, strided=True, seed=0):
    g = _gen(seed)
    td, L, S = TD[dtype], int(sum(lens)), len(lens)
    lead = (1, L) if packed else (S, L // S)
    x = torch.randn(*lead, D + (16 if strided else 0), generator=g).to(td)[..., :D]
    return dict(x=x, w=torch.randn(D, W, generator=g), bias=torch.randn(D, generator=g) if bias else None,
                state=torch.randn(S, W - 1, D, generator=g).to(td) if init else None, lens=lens, packed=packed,
                dy=torch.randn(*lead, D, generator=g).to(td), dstate_T=torch.randn(S, W - 1, D, generator=g).to(td))


def check_conv(c, silu=True, dlast=True):
    import momentum_delta_rule_gb300 as mdn
    d = _dev(c)
    D, W = d["w"].shape
    cu = torch.tensor(_cu(c["lens"]), dtype=torch.int32).cuda() if c["packed"] else None
    kw = dict(bias=d["bias"], state=d["state"], cu_seqlens=cu, activation="silu" if silu else None)
    y, last = mdn.short_conv_fwd(d["x"], d["w"], output_final_state=True, **kw)
    y2, none = mdn.short_conv_fwd(d["x"], d["w"], **kw)
    g = mdn.short_conv_bwd(d["x"], d["w"], d["dy"], dstate_T=d["dstate_T"] if dlast else None, need_dstate=True, **kw)
    again = mdn.short_conv_bwd(d["x"], d["w"], d["dy"], dstate_T=d["dstate_T"] if dlast else None, **kw)
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK and none is None and torch.equal(y, y2)
    f = lambda t: None if t is None else _np(t)
    ref, mag = (ssm.conv(f(c["x"]).reshape(-1, D), f(c["w"]), f(c["bias"]), f(c["state"]), _cu(c["lens"]), silu,
                         dy=f(c["dy"]).reshape(-1, D), dstate_T=f(c["dstate_T"]) if dlast else None, magnitude=m)
                for m in (False, True))
    _close("y", y.reshape(-1, D), ref[0], mag[0], 64)
    assert np.array_equal(last.double().cpu().numpy(), ref[1])
    L = sum(c["lens"])
    for k, v in g.items():
        if v is None:
            assert k == "dbias" and c["bias"] is None
            continue
        if again[k] is not None:
            assert torch.equal(v, again[k]), k
        _close(k, v.reshape(ref[2][k].shape), ref[2][k], mag[2][k], 64 + (L if k in ("dw", "dbias") else 0))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [0, 0, 40, 0, 1, 0, 2, 100, 0], [64, 64], [130]])
def test_conv_lengths(dtype, W, lens):
    check_conv(conv_case(dtype, lens, D=48, W=W, seed=W))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [1, 7, 8, 20, 129, 264, 2056])
def test_conv_widths(dtype, D):
    check_conv(conv_case(dtype, [19, 40], D=D, W=4, seed=D))


@pytest.mark.parametrize("kw", [dict(bias=False), dict(init=False), dict(packed=False, lens=[30, 30]), dict(strided=False)])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_options(kw, silu):
    kw = dict(dict(lens=[17, 0, 23]), **kw)
    check_conv(conv_case("bf16", D=40, W=4, seed=2, **kw), silu=silu, dlast=silu)
    check_conv(conv_case("fp32", D=40, W=3, seed=3, **kw), silu=silu, dlast=not silu)


def test_conv_many_runs():
    # more token runs than the gradient keeps partial sums for
    check_conv(conv_case("bf16", [3000, 17, 2000], D=16, W=4, seed=4))


def test_conv_without_tokens():
    import momentum_delta_rule_gb300 as mdn
    x = torch.empty(2, 0, 8, device="cuda")
    w, st = torch.randn(8, 4, device="cuda"), torch.randn(2, 3, 8, device="cuda")
    y, last = mdn.short_conv_fwd(x, w, state=st, output_final_state=True)
    assert y.shape == (2, 0, 8) and torch.equal(last, st)
    g = mdn.short_conv_bwd(x, w, y, state=st, dstate_T=st, bias=torch.zeros(8, device="cuda"))
    assert torch.equal(g["dstate"], st) and not g["dw"].any() and not g["dbias"].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,D,W", [(1, 1, 2), (5, 40, 4), (3, 129, 3), (64, 256, 4)])
def test_conv_step(dtype, n, D, W):
    import momentum_delta_rule_gb300 as mdn
    c = conv_case(dtype, [1] * n, D=D, W=W, packed=False, seed=n)
    d = _dev(c)
    want, last = mdn.short_conv_fwd(d["x"], d["w"], bias=d["bias"], state=d["state"], output_final_state=True)
    out = torch.empty_like(d["state"])
    y = mdn.short_conv_step(d["x"][:, 0], d["w"], d["state"], bias=d["bias"], state_out=out)
    st = d["state"].clone()
    y2 = mdn.short_conv_step(d["x"][:, 0], d["w"], st, bias=d["bias"])
    ref, mag = (ssm.conv(_np(c["x"]).reshape(-1, D), _np(c["w"]), _np(c["bias"]), _np(c["state"]), list(range(n + 1)),
                         magnitude=m) for m in (False, True))
    _close("y", y, ref[0], mag[0], 64)
    assert torch.equal(out, last) and torch.equal(st, last) and torch.equal(y, y2)


# ------------------------------------------------------------------- norms

def check_norm(dtype, R, D, post=True, pre=True, gate="sigmoid", scale=True, strided=True, seed=0):
    import momentum_delta_rule_gb300 as mdn
    g = _gen(seed)
    td = TD[dtype]
    rows = lambda s=1.0: (torch.randn(R, D + (8 if strided else 0), generator=g) * s).to(td)[:, :D]
    vec = lambda on: torch.randn(D, generator=g) * 0.5 + 1.0 if on else None
    c = dict(y=rows(), x=rows(2.0), gate=rows() if gate else None, w_post=vec(post), w_pre=vec(pre), scale=vec(scale),
             dx_out=rows(), dh=rows() if pre else None)
    d = _dev(c)
    kw = {k: d[k] for k in ("w_post", "w_pre", "gate", "scale")}
    kw.update(gate_act=gate or "sigmoid", eps=1e-5)
    X, h, stats = mdn.norm_residual_fwd(d["y"], d["x"], return_stats=True, **kw)
    X2, h2 = mdn.norm_residual_fwd(d["y"], d["x"], **kw)
    grads = mdn.norm_residual_bwd(d["y"], d["x"], stats, d["dx_out"], dh=d["dh"], **kw)
    again = mdn.norm_residual_bwd(d["y"], d["x"], stats, d["dx_out"], dh=d["dh"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(X, X2) and (h is None or torch.equal(h, h2))
    n = {k: _np(v) for k, v in c.items()}
    rkw = dict(w_post=n["w_post"], w_pre=n["w_pre"], gate=n["gate"], gate_act=gate or "sigmoid", scale=n["scale"], eps=1e-5)
    rX, rh, rg = ssm.norm(n["y"], n["x"], dx_out=n["dx_out"], dh=n["dh"], **rkw)
    # magnitudes: each output's terms added up as absolute values
    a = {k: None if v is None else np.abs(v) for k, v in n.items()}
    mX = ssm.norm(n["y"], np.zeros_like(n["x"]), **{**rkw, "w_pre": None})[0]
    mX = a["x"] + np.abs(mX)
    r2 = 1.0 / np.sqrt((rX * rX).mean(1, keepdims=True) + 1e-5) if pre else None
    # sums of D terms held by at least 32 threads: D / 32 + 16 roundings
    row = 64 + D / 32
    _close("x_out", X, rX, mX, row)
    if pre:
        _close("h", h, rh, mX * r2 * a["w_pre"], 2 * row)
    r1 = 1.0 / np.sqrt((n["y"] ** 2).mean(1, keepdims=True) + 1e-5) if post else 1.0
    one = np.ones(D)
    w1, w2, sc = (a[k] if a[k] is not None else one for k in ("w_post", "w_pre", "scale"))
    sig = 1 / (1 + np.exp(-n["gate"])) if gate else 1.0
    act = 1.0 if not gate else np.abs(n["gate"]) * sig if gate == "silu" else sig
    dact = 0.0 if not gate else sig * (1 + np.abs(n["gate"])) if gate == "silu" else sig
    nn = a["y"] * r1 * w1
    m = {"dx": a["dx_out"]}
    if pre:
        m["dx"] = m["dx"] + r2 * (w2 * a["dh"] + mX * r2 ** 2 * (a["dh"] * w2 * mX).mean(1, keepdims=True))
        m["dw_pre"] = (a["dh"] * mX * r2).sum(0)
    m["dscale"] = (m["dx"] * nn * act).sum(0)
    m["dgate"] = m["dx"] * sc * nn * dact
    dn = m["dx"] * sc * act
    m["dw_post"] = (dn * a["y"] * r1).sum(0)
    m["dy"] = r1 * (w1 * dn + a["y"] * r1 ** 2 * (dn * w1 * a["y"]).mean(1, keepdims=True)) if post else dn
    has = {"dy": True, "dx": True, "dgate": gate, "dw_post": post, "dw_pre": pre, "dscale": scale}
    for k, v in grads.items():
        assert (v is not None) == bool(has[k]), k
        if v is not None:
            assert torch.equal(v, again[k]), k
            _close(k, v, rg[k], m[k], 4 * row + (R if k[:2] in ("dw", "ds") else 0))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [1, 5, 8, 33, 64, 200, 1001, 1024, 2048, 4096, 5000, 8192, 16384])
def test_norm_widths(dtype, D):
    check_norm(dtype, 5, D, seed=D)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [3, 96, 130, 513, 1026, 2047, 2048, 3000, 4097, 8190, 8192, 10001, 16382, 16383, 16384])
def test_norm_widths_of_many_rows(dtype, D):
    # more rows than the kernels' small-batch shapes take
    check_norm(dtype, 640, D, gate="silu", seed=D)


@pytest.mark.parametrize("post,pre,scale", [(True, False, False), (False, True, True), (False, False, True), (True, True, False)])
@pytest.mark.parametrize("gate", [None, "sigmoid", "silu"])
def test_norm_options(post, pre, scale, gate):
    check_norm("bf16", 9, 256, post, pre, gate, scale, seed=1)
    check_norm("fp32", 3, 700, post, pre, gate, scale, strided=False, seed=2)


@pytest.mark.parametrize("dtype,D", [("bf16", 5000), ("bf16", 3001), ("fp32", 4100), ("bf16", 9001)])
@pytest.mark.parametrize("post,pre,scale,gate", [(True, False, False, "silu"), (False, True, True, None), (False, False, True, "sigmoid")])
def test_norm_options_of_wide_rows(dtype, D, post, pre, scale, gate):
    check_norm(dtype, 9, D, post=post, pre=pre, scale=scale, gate=gate, seed=D)


@pytest.mark.parametrize("R", [1, 2, 700, 5000])
def test_norm_rows(R):
    check_norm("bf16", R, 64, seed=R)
    check_norm("fp32", R, 36, gate="silu", seed=R)


def test_norm_zero_rows_and_in_place():
    import momentum_delta_rule_gb300 as mdn
    y = torch.zeros(3, 128, device="cuda")
    x = torch.randn(3, 128, device="cuda")
    x[1] = 0.0
    w = torch.ones(128, device="cuda")
    X, h, stats = mdn.norm_residual_fwd(y, x, w_post=w, w_pre=w, return_stats=True)
    assert torch.equal(X, x) and not h[1].any() and torch.isfinite(h).all()
    g = mdn.norm_residual_bwd(y, x, stats, x, dh=x, w_post=w, w_pre=w)
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None)
    keep = x.clone()
    X2, h2 = mdn.norm_residual_fwd(y + 1, keep, w_post=w, w_pre=w, x_out=keep)
    X3, h3 = mdn.norm_residual_fwd(y + 1, x, w_post=w, w_pre=w)
    assert X2 is keep and torch.equal(X2, X3) and torch.equal(h2, h3)
    e = torch.empty(0, 128, device="cuda")
    X, h, stats = mdn.norm_residual_fwd(e, e, w_post=w, w_pre=w, return_stats=True)
    g = mdn.norm_residual_bwd(e, e, stats, e, dh=e, w_post=w, w_pre=w)
    assert X.shape == (0, 128) and not g["dw_post"].any() and not g["dw_pre"].any()


# ---------------------------------------------------------- streams, graphs

def test_calls_on_another_stream_and_in_a_graph():
    import momentum_delta_rule_gb300 as mdn
    c = _dev(scan_case("bf16", [70, 0, 33], D=64, N=16, seed=31))
    args, kw = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"]), _scan_kw(c)
    w = torch.randn(64, 4, device="cuda")
    ones = torch.ones(64, device="cuda")

    def layer(stream=None):
        x, _ = mdn.short_conv_fwd(c["u"], w, cu_seqlens=kw["cu_seqlens"], stream=stream)
        y, hT, hc = mdn.ssm_scan_fwd(x, *args[1:], h0=c["h0"], return_chunk_states=True, stream=stream, **kw)
        X, h, st = mdn.norm_residual_fwd(y, x, w_post=ones, w_pre=ones, return_stats=True, stream=stream)
        n = mdn.norm_residual_bwd(y, x, st, X, dh=h, w_post=ones, w_pre=ones, stream=stream)
        g = mdn.ssm_scan_bwd(x, *args[1:], hc, n["dy"], stream=stream, **kw)
        v = mdn.short_conv_bwd(c["u"], w, g["du"], cu_seqlens=kw["cu_seqlens"], stream=stream)
        return [y, hT, X, h, n["dw_post"], g["dA"], g["dB"], g["ddt"], v["dx"], v["dw"]]

    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert mdn.device_status() == mdn.MDN_OK
