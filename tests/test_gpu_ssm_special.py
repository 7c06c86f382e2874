"""Infinities and NaN in the operators' inputs: where the definition gives a
finite number, an infinity or NaN, so do the kernels.  Numbers of states that
fill no whole lanes, lengths that fill no whole batch of tokens and the places
behind them must not turn an infinity into NaN, or a finite number into either.
Finite values have the tolerances of ``tests/test_gpu_ssm.py``."""
import numpy as np
import pytest
import torch

from oracle import ssm
from tests.test_gpu_ssm import TD, _dev, _gen, _np, _scan_kw, _scan_ref, conv_case, scan_case

pytestmark = pytest.mark.gpu

INF = float("inf")
STATES = [1, 2, 3, 4, 5, 8, 12, 16, 20, 24, 33, 64, 100, 128]


def _same_kind(name, got, ref, mag, ulps):
    """Finite where ref is and near it, the same infinity, NaN or infinite for NaN."""
    eps = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy().reshape(ref.shape)
    fin = np.isfinite(ref)
    with np.errstate(all="ignore"):
        tol = eps * np.abs(ref) + (1 + eps) * ulps * 2.0 ** -24 * np.abs(mag) + 1e-37
        tol = np.where(np.isfinite(tol), tol, np.finfo(np.float32).max)
        bad = np.where(fin, ~(np.abs(g - ref) <= tol), np.where(np.isnan(ref), np.isfinite(g), g != ref))
    at = np.argwhere(bad)
    assert not len(at), "%s: %d of %d, first at %s: %s for %s" % (name, len(at), bad.size, at[0], g[tuple(at[0])],
                                                                  ref[tuple(at[0])])


def positive_case(dtype, N, G=1, lens=(7, 34), D=12, seed=0):
    """Every term of every sum positive (but A): an infinity is not met by its opposite."""
    c = scan_case(dtype, list(lens), D=D, N=N, G=G, strided=False, seed=seed)
    for k in ("u", "Bm", "Cm", "z", "h0", "D_skip"):
        c[k] = c[k].abs() + 0.125
    return c


def check_kind(c, dy_at=None, dh_at=None):
    import momentum_delta_rule_gb300 as mdn
    d = _dev(c)
    D = d["A"].shape[0]
    args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"])
    y, hT, hc = mdn.ssm_scan_fwd(*args, h0=d["h0"], return_chunk_states=True, **_scan_kw(d))
    dy = (torch.rand(y.shape, generator=_gen(1)) + 0.125).to(y.dtype)
    dhT = torch.rand(hT.shape, generator=_gen(2)) + 0.125
    if dy_at is not None:
        dy[dy_at] = INF
    if dh_at is not None:
        dhT[dh_at] = INF
    g = mdn.ssm_scan_bwd(*args, hc, dy.cuda(), dh_T=dhT.cuda(), need_dh0=True, **_scan_kw(d))
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        ref, mag = (_scan_ref(c, dy=_np(dy).reshape(-1, D), dh_T=_np(dhT), magnitude=m) for m in (False, True))
    T, L = max(c["lens"]), sum(c["lens"])
    _same_kind("y", y, ref[0], mag[0], 64 + 16 * T)
    _same_kind("h_T", hT, ref[1], mag[1], 64 + 16 * T)
    for k, v in g.items():
        _same_kind(k, v, ref[3][k], mag[3][k], 2 * (64 + 16 * T) + max(L, D))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_infinite_input(dtype, N):
    # in the middle of a sequence, and as its last token
    c = positive_case(dtype, N, seed=N)
    c["u"][0, 3, 2] = INF
    c["u"][0, 40, 5] = INF
    check_kind(c)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_infinite_adjoint_of_the_final_state(dtype, N):
    check_kind(positive_case(dtype, N, seed=N), dh_at=(0, 4, N - 1))
    check_kind(positive_case(dtype, N, seed=N), dh_at=(1, 9, 0))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_infinite_step(dtype, N):
    c = positive_case(dtype, N, seed=N)
    c["dt"][0, 4, 1] = INF
    c["dt"][0, 40, 7] = INF
    check_kind(c)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_infinite_adjoint(dtype, N):
    check_kind(positive_case(dtype, N, seed=N), dy_at=(0, 30, 3))
    check_kind(positive_case(dtype, N, G=2, D=14, seed=N), dy_at=(0, 6, 9))


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("N", [16, 20])
def test_infinite_states_of_cut_sequences(N, packed):
    # a segment's decay is zero in fp32 where none of its tokens' is
    c = positive_case("fp32", N, lens=[700], seed=N)
    c["packed"] = packed
    c["A"] = c["A"].clamp(-2.0, 0.0) - 20.0
    c["dt_bias"].zero_()
    u = c["u"].clone()
    c["u"][0, 100, 4] = INF
    check_kind(c)
    c["u"] = u
    check_kind(c, dy_at=(0, 600, 7))
    check_kind(c, dh_at=(0, 2, 1))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_infinite_step_of_one_token(dtype, N):
    import momentum_delta_rule_gb300 as mdn
    c = positive_case(dtype, N, lens=[1] * 3, D=40, seed=N)
    c["u"][0, 0, 2] = INF
    c["u"][0, 1, 35] = INF
    c["dt"][0, 2, 17] = INF
    d = _dev(c)
    kw = {k: d[k] for k in ("D_skip", "dt_bias", "softplus")}
    h = d["h0"].clone()
    y = mdn.ssm_scan_step(d["u"][0], d["dt"][0], d["A"], d["Bm"][0], d["Cm"][0], h, z=d["z"][0], **kw)
    with np.errstate(all="ignore"):
        ref, mag = (_scan_ref(c, magnitude=m) for m in (False, True))
    _same_kind("y", y, ref[0], mag[0], 80 + N)
    _same_kind("h", h, ref[1], mag[1], 80)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,lens", [(16, [5, 33, 64, 1, 6, 2]), (3, [5, 33, 64, 1, 6, 2]), (20, [7, 31, 4]), (128, [9, 2]),
                                    (16, [1501]), (8, [1403, 30])])
def test_states_that_decay_at_once(dtype, N, lens):
    # A = -inf: exp(delta A) = 0 for every step, as of a very negative A
    import momentum_delta_rule_gb300 as mdn
    c = scan_case(dtype, lens, D=24, N=N, seed=N)
    c["A"][::2, ::3] = -1e30
    ref, mag = _scan_ref(c), _scan_ref(c, magnitude=True)
    d = _dev(c)
    dy, dhT = torch.randn(1, sum(lens), 24, generator=_gen(1)).to(d["u"].dtype).cuda(), torch.ones_like(d["h0"])

    def run():
        args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"])
        y, hT, hc = mdn.ssm_scan_fwd(*args, h0=d["h0"], return_chunk_states=True, **_scan_kw(d))
        slots = sum((n + 31) // 32 for n in lens)
        g = mdn.ssm_scan_bwd(*args, hc, dy, dh_T=dhT, need_dh0=True, **_scan_kw(d))
        h = d["h0"].clone()
        n = len(lens)
        kw = {k: d[k] for k in ("D_skip", "dt_bias", "softplus")}
        ys = mdn.ssm_scan_step(d["u"][0, :n], d["dt"][0, :n], d["A"], d["Bm"][0, :n], d["Cm"][0, :n], h, **kw)
        return [y, hT, hc[:slots], ys, h] + [v for v in g.values() if v is not None]

    want = run()
    _same_kind("y", want[0], ref[0], mag[0], 64 + 16 * max(lens))
    _same_kind("h_T", want[1], ref[1], mag[1], 64 + 16 * max(lens))
    d["A"][::2, ::3] = -INF
    got = run()
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


NAN = float("nan")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [3, 16, 20])
@pytest.mark.parametrize("key,at", [("u", (0, 3, 2)), ("u", (0, 40, 5)), ("dt", (0, 6, 0)), ("Bm", (0, 9, 0, 1)),
                                    ("Cm", (0, 40, 0, 2)), ("z", (0, 20, 3)), ("h0", (1, 4, 0))])
def test_nan_goes_no_further_than_in_the_formulas(dtype, N, key, at):
    c = scan_case(dtype, [7, 34], D=12, N=N, strided=False, seed=N)
    c[key][at] = NAN
    check_kind(c)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("at", [6, 7, 40])
def test_nan_adjoint_goes_no_further_than_in_the_formulas(dtype, at):
    import momentum_delta_rule_gb300 as mdn
    c = scan_case(dtype, [7, 34], D=12, N=20, strided=False, seed=at)
    d = _dev(c)
    args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"])
    dy = torch.randn(1, 41, 12, generator=_gen(at)).to(d["u"].dtype)
    dy[0, at, 5] = NAN
    hc = mdn.ssm_scan_fwd(*args, h0=d["h0"], return_chunk_states=True, **_scan_kw(d))[2]
    g = mdn.ssm_scan_bwd(*args, hc, dy.cuda(), need_dh0=True, **_scan_kw(d))
    ref, mag = (_scan_ref(c, dy=_np(dy).reshape(-1, 12), magnitude=m) for m in (False, True))
    for k, v in g.items():
        _same_kind(k, v, ref[3][k], mag[3][k], 2 * (64 + 16 * 34) + 41)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [48, 46, 47])
@pytest.mark.parametrize("value", [NAN, INF])
def test_convolution_of_nan_and_infinities(dtype, D, value):
    import momentum_delta_rule_gb300 as mdn
    lens = [5, 1, 0, 30, 16]
    cu = [0] + np.cumsum(lens).tolist()
    c = conv_case(dtype, lens, D=D, W=4, strided=False, seed=D)
    for t, ch in ((4, 3), (5, 7), (35, 9), (36, 11), (15, 2), (51, 20)):      # ends, starts, middles
        c["x"][0, t, ch] = value
    c["dy"][0, 35, 30] = c["dy"][0, 6, 31] = value
    d = _dev(c)
    kw = dict(bias=d["bias"], state=d["state"], cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    y, last = mdn.short_conv_fwd(d["x"], d["w"], output_final_state=True, **kw)
    g = mdn.short_conv_bwd(d["x"], d["w"], d["dy"], dstate_T=d["dstate_T"], **kw)
    with np.errstate(all="ignore"):
        ref, mag = (ssm.conv(_np(c["x"])[0], _np(c["w"]), _np(c["bias"]), _np(c["state"]), cu, dy=_np(c["dy"])[0],
                             dstate_T=_np(c["dstate_T"]), magnitude=m) for m in (False, True))
    _same_kind("y", y, ref[0], mag[0], 64)
    _same_kind("state_T", last, ref[1], np.abs(ref[1]), 0)
    for k, v in g.items():
        _same_kind(k, v, ref[2][k], mag[2][k], 64 + sum(lens))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 1001, 5000])
@pytest.mark.parametrize("value", [NAN, INF])
def test_norms_of_nan_and_infinities(dtype, D, value):
    # a row has its own sums: the others', and the rows behind it, stay
    import momentum_delta_rule_gb300 as mdn
    R, bad = 400, 131
    g = _gen(D)
    y, x, gate, dX, dh = (torch.randn(R, D, generator=g).to(TD[dtype]).cuda() for _ in range(5))
    w = torch.rand(D, generator=g).cuda() + 0.5
    kw = dict(w_post=w, w_pre=w, scale=w, gate=gate)

    def run():
        X, h, st = mdn.norm_residual_fwd(y, x, return_stats=True, **kw)
        b = mdn.norm_residual_bwd(y, x, st, dX, dh=dh, **kw)
        return [X, h, st, b["dy"], b["dx"], b["dgate"]]

    want = run()
    for t in (y, x, gate, dX, dh):
        keep = t[bad].clone()
        t[bad, D // 2] = value
        got = run()
        t[bad] = keep
        for a, b in zip(got, want):
            assert torch.equal(a[:bad], b[:bad]) and torch.equal(a[bad + 1:], b[bad + 1:])
