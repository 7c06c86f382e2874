"""GPU parity of the group norm with an activation against the fp64 reference
(``oracle/attn.py``).

Tolerances.  Let a group have N elements, mean a, deviation s, x its largest
|x - a| / s (the largest |n|), and r = |a| / s.  In fp32 (u = 2^-24):
  * sums over a group make at most N roundings, in fact one for each of a
    thread's at most 512 terms and one a level of joining: J = min(N, 512) + 32;
  * the mean is off by J u (|a| + s), n by (J (1 + r) + J (1 + x) + 8) u (1 + x):
    E_n = J (2 + r + x) (1 + x) u covers it;
  * u = n w + b is off by E_n |w| + 2 u (|n w| + |b|), activations and their
    derivatives are 1.1-Lipschitz and take ex2 and rcp of 2^-22 each: 16 u;
  * the gradient's means are means of terms each off by that much, and the
    parameters' sums have at most as many roundings as tokens, in order.
An output adds half a step of its type.
"""
import numpy as np
import pytest
import torch

from oracle import attn

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def case(dtype, lens, D, G, gate=True, activation="silu", over="token", center=True, affine=True, packed=True, offset=0,
         pad=0, mean=0.3, std=1.5, seed=0):
    g = torch.Generator().manual_seed(seed)
    L, S = int(sum(lens)), len(lens)
    lead = (1, L) if packed else (S, L // S)
    rn = lambda *s: torch.randn(s, generator=g)
    wide = (rn(*lead, offset + 2 * D + pad) * std + mean).to(TD[dtype])
    return dict(x=wide[..., offset:offset + D], gate=wide[..., offset + D:offset + 2 * D] if gate else None,
                weight=1 + 0.2 * rn(D) if affine else None, bias=0.2 * rn(D) if affine else None,
                dy=rn(*lead, D).to(TD[dtype]), groups=G, activation=activation, over=over, center=center, lens=lens,
                packed=packed)


def dev(c):
    out, moved = {}, {}
    for k, v in c.items():
        if isinstance(v, torch.Tensor):
            base = v._base if v._base is not None else v
            if id(base) not in moved:
                moved[id(base)] = base.cuda()
            v = torch.as_strided(moved[id(base)], v.shape, v.stride(), v.storage_offset())
        out[k] = v
    seq = c["over"] == "sequence" and c["packed"]
    out["cu"] = torch.tensor([0] + list(np.cumsum(c["lens"])), dtype=torch.int32).cuda() if seq else None
    return out


def run(d):
    import momentum_delta_rule_gb300 as mdn
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], activation=d["activation"], over=d["over"],
              center=d["center"], cu_seqlens=d["cu"])
    y, stats = mdn.group_norm_fwd(d["x"], d["groups"], return_stats=True, **kw)
    assert torch.equal(y, mdn.group_norm_fwd(d["x"], d["groups"], **kw))
    return dict(y=y, stats=stats, **mdn.group_norm_bwd(d["x"], d["groups"], stats, d["dy"], **kw))


def check(c, got):
    D, G = c["x"].shape[-1], c["groups"]
    L = c["x"].numel() // D
    f = lambda t: None if t is None else _np(t).reshape(L, D)
    cu = [0] + list(np.cumsum(c["lens"])) if c["over"] == "sequence" else None
    x, dy, gate = f(c["x"]), f(c["dy"]), f(c["gate"])
    w = _np(c["weight"]) if c["weight"] is not None else np.ones(D)
    b = _np(c["bias"]) if c["bias"] is not None else np.zeros(D)
    y, stats, g = attn.group_norm(x, G, _np(c["weight"]), _np(c["bias"]), gate, c["activation"], cu, c["center"], 1e-5, dy)
    runs = [(t, t + 1) for t in range(L)] if cu is None else list(zip(cu[:-1], cu[1:]))
    per = lambda i, a, e: np.repeat(stats[i], D // G, axis=0)
    mean, r = np.zeros((L, D)), np.zeros((L, D))
    for i, (a, e) in enumerate(runs):
        s = np.repeat(stats[i], D // G, axis=0)
        mean[a:e], r[a:e] = s[:, 0], s[:, 1]
    n = (x - mean) * r

    def largest(t):
        """The largest |t| of each element's group."""
        out = np.zeros((L, D))
        for a, e in runs:
            if e > a:
                m = np.abs(t[a:e]).reshape(e - a, G, -1).max((0, 2))
                out[a:e] = np.repeat(m, D // G)
        return out

    N = max([e - a for a, e in runs] or [0]) * (D // G)
    J = min(N, 512) + 32
    big = largest(n)
    En = J * (2 + np.abs(mean) * r + big) * (1 + big) * U
    u = n * w + b
    Eu = En * np.abs(w) + 2 * U * (np.abs(n * w) + np.abs(b))
    if gate is None:
        a, da, dd = attn.act(u, c["activation"])
        Ey = 1.1 * Eu + 16 * U * np.abs(u)
        du, Edu = dy * da, np.abs(dy) * (dd * Eu + 16 * U * (1 + np.abs(u)))
    else:
        a, da, _ = attn.act(gate, c["activation"])
        Ey = Eu * np.abs(a) + 16 * U * np.abs(u * a)
        du, Edu = dy * a, 16 * U * np.abs(dy * a)
    dn, Edn = du * w, Edu * np.abs(w) + U * np.abs(du * w)
    mdn_, mdnn = largest(dn), largest(dn * n)
    Emean = J * U * (mdn_ + mdnn * (1 + big)) + largest(Edn) * (1 + big * (1 + big)) + largest(dn) * largest(En) * (1 + big)
    tol = dict(y=Ey, dx=r * (Edn + Emean + largest(dn * n) * En + 8 * U * (np.abs(dn) + mdn_ + big * mdnn)
                             + (np.abs(dn) + mdn_ + big * mdnn) * En),
               dw=(np.abs(du) * En + Edu * np.abs(n)).sum(0) + (L + 8) * U * np.abs(du * n).sum(0),
               dbias=Edu.sum(0) + (L + 8) * U * np.abs(du).sum(0))
    if gate is not None:
        tol["dgate"] = np.abs(dy * da) * Eu + 16 * U * np.abs(dy * u) * (np.abs(da) + 1)
    ref = dict(y=y, **g)
    for name, t in tol.items():
        if got[name] is None:
            assert name in ("dw", "dbias") and c["weight"] is None
            continue
        eps = torch.finfo(got[name].dtype).eps / 2
        v = got[name].double().cpu().numpy().reshape(ref[name].shape)
        assert np.isfinite(v).all(), name
        t = eps * np.abs(ref[name]) + (1 + eps) * t + 1e-37
        off = np.abs(v - ref[name])
        assert (off <= t).all(), "%s: %d of %d off, worst %.2f times the tolerance" % (
            name, (off > t).sum(), off.size, (off / t).max())
        if v.size >= 4096:
            miss, size = np.linalg.norm(v - ref[name]), np.linalg.norm(ref[name])
            # (fp32: a mean is at best the number next to it, half a step 2^-24
            # |a| off, which moves every n of its group by r 2^-24; sums of J <
            # 2^8 terms in a row stay within that many of those)
            far = 1 + (np.abs(mean) * r).max()
            assert miss <= (2.0 ** -8 if got[name].dtype == torch.bfloat16 else 2.0 ** -16 * far) * size, (name, miss, size)


def check_case(c):
    import momentum_delta_rule_gb300 as mdn
    d = dev(c)
    got, again = run(d), run(d)
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    for name in got:
        assert got[name] is None or torch.equal(got[name], again[name]), name
    check(c, got)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,D,G", [(1, 1, 1), (3, 8, 8), (70, 2048, 16), (33, 1001, 7), (5, 330, 6), (129, 64, 1),
                                      (9, 2048, 2), (4, 4096, 1), (3, 16384, 1), (3, 16383, 3), (2, 8190, 1),
                                      (700, 96, 12), (41, 40, 10), (20, 6, 3), (3000, 128, 2), (6, 9216, 2)])
def test_groups_of_a_token(dtype, rows, D, G):
    check_case(case(dtype, [rows], D, G, seed=rows))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rows,D,G", [(650, 2049, 1), (330, 4098, 2), (400, 4608, 1), (310, 2438, 1), (700, 1536, 1)])
def test_wide_groups_of_more_tokens_than_blocks(dtype, gate, rows, D, G):
    check_case(case(dtype, [rows], D, G, gate, seed=rows))


SEQS = [([1], 4, 2, True), ([64, 64], 64, 4, False), ([5, 0, 130, 1], 330, 6, True), ([700], 96, 1, True),
        ([33, 33, 33], 2048, 32, False), ([40, 3], 1001, 7, True), ([300, 20], 16, 16, True), ([9, 2], 16384, 1, True),
        ([7], 8190, 2, True), ([2100, 900], 40, 5, True)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,D,G,packed", SEQS)
def test_groups_of_a_sequence(dtype, lens, D, G, packed):
    check_case(case(dtype, lens, D, G, over="sequence", packed=packed, gate=len(lens) % 2 == 0, seed=D))


@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("center,affine", [(True, True), (False, True), (True, False), (False, False)])
def test_options(over, activation, gate, center, affine):
    check_case(case("fp32", [37, 90], 64, 4, gate, activation, over, center, affine, seed=3))


@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("dtype,offset,pad", [("bf16", 1, 0), ("bf16", 2, 4), ("bf16", 8, 8), ("fp32", 1, 0), ("fp32", 4, 4)])
def test_rows_of_any_alignment(over, dtype, offset, pad):
    check_case(case(dtype, [50, 31], 128, 2, over=over, offset=offset, pad=pad, seed=11))


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_a_mean_far_from_zero(over):
    """The deviations are taken from the mean, not from sums of squares."""
    check_case(case("fp32", [200], 256, 4, over=over, mean=1000.0, std=1.0))


def test_constant_groups():
    import momentum_delta_rule_gb300 as mdn
    for over in ("token", "sequence"):
        x = torch.full((2, 30, 16), 3.0, device="cuda")
        y, stats = mdn.group_norm_fwd(x, 4, over=over, return_stats=True, bias=torch.ones(16, device="cuda"))
        assert (y == 1).all() and (stats[..., 0] == 3).all()


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 70, 100], [0, 50, 70, 99], [0, -5, 70, 100], [0, 2000000000, 70, 100]])
def test_malformed_sequences_leave_outputs_alone(cu):
    import momentum_delta_rule_gb300 as mdn
    d = dev(case("bf16", [40, 30, 30], 64, 4, over="sequence"))
    good = run(d)
    bad = torch.tensor(cu, dtype=torch.int32).cuda()
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], activation="silu", over="sequence", cu_seqlens=bad)
    y = torch.full((1, 100, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, stats = mdn.group_norm_fwd(d["x"], 4, y=y, return_stats=True, **kw)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert (y == 7).all() and (stats == 0).all()
    g = mdn.group_norm_bwd(d["x"], 4, good["stats"], d["dy"], **kw)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert (g["dw"] == 0).all() and (g["dbias"] == 0).all()


def test_no_rows():
    import momentum_delta_rule_gb300 as mdn
    for over in ("token", "sequence"):
        x, w = torch.zeros(2, 0, 16, device="cuda"), torch.ones(16, device="cuda")
        y, stats = mdn.group_norm_fwd(x, 4, weight=w, over=over, return_stats=True)
        assert y.shape == x.shape and (stats == 0).all()
        g = mdn.group_norm_bwd(x, 4, stats, x, weight=w, bias=w, over=over)
        assert (g["dw"] == 0).all() and (g["dbias"] == 0).all()


def test_nan_and_infinities_stay_in_their_group():
    import momentum_delta_rule_gb300 as mdn
    for bad in (float("nan"), float("inf")):
        for over in ("token", "sequence"):
            d = dev(case("fp32", [40, 30], 64, 4, over=over))
            kw = dict(gate=d["gate"], activation="silu", over=over, cu_seqlens=d["cu"])
            want = mdn.group_norm_fwd(d["x"], 4, **kw)
            d["x"][0, 10, 20] = bad
            got = mdn.group_norm_fwd(d["x"], 4, **kw)
            rows = slice(10, 11) if over == "token" else slice(0, 40)
            assert got[0, rows, 16:32].isnan().all()
            got[0, rows, 16:32] = want[0, rows, 16:32]
            assert torch.equal(got, want)


def test_streams_and_graphs():
    import momentum_delta_rule_gb300 as mdn
    for over in ("token", "sequence"):
        d = dev(case("bf16", [300, 80], 128, 4, over=over))
        want = run(d)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y = mdn.group_norm_fwd(d["x"], 4, d["weight"], d["bias"], d["gate"], "silu", over, cu_seqlens=d["cu"], stream=side)
        side.synchronize()
        assert torch.equal(y, want["y"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run_unchecked(d)
        for t in got.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name in got:
            assert torch.equal(got[name], want[name]), name


def run_unchecked(d):
    import momentum_delta_rule_gb300 as mdn
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], activation=d["activation"], over=d["over"],
              center=d["center"], cu_seqlens=d["cu"])
    y, stats = mdn.group_norm_fwd(d["x"], d["groups"], return_stats=True, **kw)
    return dict(y=y, stats=stats, **mdn.group_norm_bwd(d["x"], d["groups"], stats, d["dy"], **kw))


def test_workspaces_hold_what_is_written():
    import momentum_delta_rule_gb300 as mdn
    for over, lens, D, G in (("token", [500], 96, 12), ("sequence", [300, 200], 330, 6), ("token", [2], 16383, 16383)):
        d = dev(case("bf16", lens, D, G, over=over))
        want = run(d)
        L, n = sum(lens), len(lens) if over == "sequence" else 1
        kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], activation="silu", over=over, cu_seqlens=d["cu"])
        for name in ("fwd", "bwd"):
            need = getattr(mdn.lib(), "mdn_group_norm_%s_workspace_size" % name)(n, L, D, G, over == "sequence", mdn.MDN_BF16)
            ws = torch.full((need + 4096,), 0x55, dtype=torch.uint8, device="cuda")
            if name == "fwd":
                assert torch.equal(mdn.group_norm_fwd(d["x"], G, workspace=ws[:need], **kw), want["y"])
            else:
                g = mdn.group_norm_bwd(d["x"], G, want["stats"], d["dy"], workspace=ws[:need], **kw)
                assert torch.equal(g["dw"], want["dw"]) and torch.equal(g["dx"], want["dx"])
            assert (ws[need:] == 0x55).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_sequences(dtype):
    check_case(case(dtype, [(7 * i) % 4 for i in range(1500)], 48, 3, over="sequence", seed=17))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,D,G,packed", [([9000], 64, 1, True), ([4001, 3000], 96, 2, True), ([5000, 5000], 40, 1, False),
                                             ([40000], 16, 2, False)])
def test_long_sequences(dtype, lens, D, G, packed):
    """Beyond what a cluster's shared memory holds, and just within."""
    check_case(case(dtype, lens, D, G, over="sequence", packed=packed, seed=19))


def test_a_malformed_end_of_many_sequences():
    import momentum_delta_rule_gb300 as mdn
    x = torch.randn(1, 3000, 32, device="cuda")
    cu = torch.arange(0, 3001, 2, dtype=torch.int32, device="cuda")
    cu[700] = 5
    y = torch.full_like(x, 7.0)
    _, stats = mdn.group_norm_fwd(x, 4, over="sequence", cu_seqlens=cu, y=y, return_stats=True)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert (y == 7).all() and (stats == 0).all()
