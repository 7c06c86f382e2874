"""GPU parity of linear attention with a decay for each head against the fp64
reference (``oracle/attn.py``), element by element.

Tolerance of an output x with the magnitude m of its terms (the reference
formula over absolute values): half a step of its type, eps / 2 |x|, plus the
evaluation's own error.  That is
  * fp32 sums: at most one rounding a term, of which a product chain has dk or
    dv in q k^T (or do v^T), 64 within a chunk, T + T / 64 along the state and
    dk or dv where the state is read, and 16 for the decay's exp2 and the
    products: U = 2 (dk + dv) + 2 T + 80 times 2^-24 m;
  * the decays' exponents e log2(lambda): log2(e) log_decay and its product with
    e are rounded, each by 2^-24 relative (and log2(e) itself): 4 2^-24 covers
    the three; the reference is evaluated again with decays that much larger;
  * operands that are not fp32: bf16 rows round q k^T with its decay to bf16, or
    the state, of which each term passes one: half a step, 2^-8 m.  The states
    themselves are sums of products with v (or do) times a decay, as two bf16
    parts: the decay's leave 2^-17 of it, the second part of the product is
    rounded by half a step of at most 2^-8 of it, 2^-16: 3 2^-17 m.  (fp32 rows are products of three bf16 parts each, which
    leave out less than a rounding in fp32.)
"""
import numpy as np
import pytest
import torch

from oracle import attn

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def case(dtype, lens, H, Hkv, dk, dv, packed=True, init=True, offset=0, pad=0, scale=None, decay=None, seed=0):
    """Inputs on the CPU; q, k and v lie side by side `pad` elements apart, the
    first `offset` elements into the rows."""
    g = torch.Generator().manual_seed(seed)
    L, S = int(sum(lens)), len(lens)
    lead = (1, L) if packed else (S, L // S)
    widths = [H * dk, Hkv * dk, Hkv * dv]
    wide = torch.randn(*lead, offset + sum(widths) + 3 * pad, generator=g).to(TD[dtype])
    parts, at = [], offset
    for w in widths:
        parts.append(wide[..., at:at + w])
        at += w + pad
    q, k, v = (t.unflatten(-1, (-1, d)) for t, d in zip(parts, (dk, dk, dv)))
    rn = lambda *s: torch.randn(s, generator=g)
    return dict(q=q, k=k, v=v, log_decay=-torch.exp2(-8 * torch.rand(H, generator=g)) if decay is None else torch.tensor(decay),
                S0=rn(S, H, dk, dv) if init else None, do=rn(*lead, H, dv).to(TD[dtype]), dS_T=rn(S, H, dk, dv),
                scale=dk ** -0.5 if scale is None else scale, lens=lens, packed=packed)


def dev(c):
    """The case on the GPU, slices staying slices of one wider tensor."""
    out, moved = {}, {}
    for k, v in c.items():
        if isinstance(v, torch.Tensor):
            base = v._base if v._base is not None else v
            if id(base) not in moved:
                moved[id(base)] = base.cuda()
            v = torch.as_strided(moved[id(base)], v.shape, v.stride(), v.storage_offset())
        out[k] = v
    out["cu"] = torch.tensor([0] + list(np.cumsum(c["lens"])), dtype=torch.int32).cuda() if c["packed"] else None
    return out


def reference(c, **kw):
    L = int(sum(c["lens"]))
    f = lambda t: _np(t).reshape(L, *t.shape[2:])
    return attn.linear_attn(f(c["q"]), f(c["k"]), f(c["v"]), _np(c["log_decay"]), c["scale"], _np(c["S0"]),
                            [0] + list(np.cumsum(c["lens"])), do=f(c["do"]), dS_T=_np(c["dS_T"]), **kw)


def flat(r):
    return dict(o=r[0], S_T=r[1], **r[2])


def check(c, got):
    ref, mag = flat(reference(c)), flat(reference(c, magnitude=True))
    late = flat(reference(c, magnitude=True, exponent_error=4 * 2.0 ** -24))
    T, (dk, dv) = max(c["lens"]), (c["q"].shape[-1], c["v"].shape[-1])
    U = (2 * (dk + dv) + 2 * T + 80) * 2.0 ** -24
    for name, x in got.items():
        if x is None:
            continue
        eps = torch.finfo(x.dtype).eps / 2
        g = x.double().cpu().numpy().reshape(ref[name].shape)
        assert np.isfinite(g).all(), name
        state = name in ("S_T", "dS0")
        mixed = (3 * 2.0 ** -17 if state else 2.0 ** -8 + 3 * 2.0 ** -17) if c["q"].dtype == torch.bfloat16 else 0.0
        tol = eps * np.abs(ref[name]) + (1 + eps) * ((U + mixed) * mag[name] + (late[name] - mag[name])) + 1e-37
        bad = np.abs(g - ref[name]) > tol
        worst = float((np.abs(g - ref[name]) / tol).max()) if g.size else 0.0
        assert not bad.any(), "%s: %d of %d off, worst %.2f times the tolerance, at %s" % (
            name, bad.sum(), bad.size, worst, np.argwhere(bad)[:3].tolist())
        # and as a whole: three roundings to bf16 at most, each at most 2^-8 of
        # its value and uniform within (2^-8 / sqrt 3), on terms that add up in
        # squares; sums of 2^-24 and parts of 3 2^-17 at most stay below 2^-15
        if x.numel() >= 4096:
            off, size = np.linalg.norm(g - ref[name]), np.linalg.norm(ref[name])
            assert off <= (2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -15) * size, (name, off, size)


def run(d, train=True):
    import momentum_delta_rule_gb300 as mdn
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    kw = dict(scale=d["scale"], S0=d["S0"], cu_seqlens=d["cu"])
    o, S_T = mdn.linear_attn_fwd(*args, **kw)
    out = dict(o=o, S_T=S_T)
    if train:
        out.update(mdn.linear_attn_bwd(*args, d["do"], dS_T=d["dS_T"], need_dS0=True, **kw))
    return out


def check_case(c):
    import momentum_delta_rule_gb300 as mdn
    d = dev(c)
    got, again = run(d), run(d)
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    for name in got:
        assert torch.equal(got[name], again[name]), name
    check(c, got)


SHAPES = [
    # lens, H, Hkv, dk, dv, packed
    ([1], 1, 1, 1, 1, False),
    ([1, 1, 1], 2, 2, 64, 64, False),
    ([64, 64], 2, 2, 64, 64, False),
    ([130, 130], 2, 1, 128, 128, False),
    ([63, 0, 65, 1, 128, 200], 3, 3, 128, 128, True),
    ([0, 5, 0], 2, 2, 32, 48, True),
    ([70, 129], 4, 2, 128, 64, True),
    ([70, 129], 4, 1, 64, 128, True),
    ([100], 2, 2, 16, 96, False),
    ([77, 3], 2, 2, 114, 40, True),
    ([77, 66], 3, 1, 57, 33, True),
    ([191], 1, 1, 127, 1, False),
    ([191], 1, 1, 2, 128, False),
    ([90, 100], 2, 2, 72, 72, True),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed", SHAPES)
def test_shapes(dtype, lens, H, Hkv, dk, dv, packed):
    check_case(case(dtype, lens, H, Hkv, dk, dv, packed, seed=len(lens) + dk))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed", [
    ([2500], 2, 1, 32, 32, False),
    ([1700, 1700], 1, 1, 128, 64, False),
    ([1100, 3, 0, 3300], 2, 2, 16, 24, True),
    ([64 * 40], 1, 1, 64, 128, False),
])
def test_long_sequences(dtype, lens, H, Hkv, dk, dv, packed):
    check_case(case(dtype, lens, H, Hkv, dk, dv, packed, seed=5))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("offset,pad,dk,dv", [(0, 8, 64, 64), (1, 0, 64, 64), (2, 0, 128, 64), (0, 1, 64, 128),
                                              (0, 2, 40, 72), (4, 4, 128, 128)])
def test_rows_of_any_alignment(dtype, offset, pad, dk, dv):
    check_case(case(dtype, [66, 131], 2, 2, dk, dv, True, offset=offset, pad=pad, seed=7))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("decay", [[0.0, 0.0], [-1e-4, -0.5], [-3.0, -40.0], [-float("inf"), -1e-30]])
def test_decays(dtype, decay):
    c = case(dtype, [150, 65], 2, 2, 64, 64, True, decay=decay, seed=9)
    if decay[0] == -float("inf"):
        c["log_decay"] = torch.tensor([-300.0, decay[1]])    # the reference's l |log l| stays finite; both are zero
    d = dev(c)
    d["log_decay"] = torch.tensor(decay).cuda()
    got = run(d)
    torch.cuda.synchronize()
    check(c, got)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_without_states(dtype):
    import momentum_delta_rule_gb300 as mdn
    c = case(dtype, [100, 100], 2, 2, 64, 64, False, init=False, scale=-0.25)
    c["dS_T"] = torch.zeros_like(c["dS_T"])
    d = dev(c)
    o, S_T = mdn.linear_attn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=d["scale"], output_final_state=False)
    assert S_T is None
    g = mdn.linear_attn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=d["scale"])
    assert g["dS0"] is None
    torch.cuda.synchronize()
    check(c, dict(o=o, **g))


def test_a_scale_of_zero():
    c = case("bf16", [70], 1, 1, 64, 64, True, scale=0.0)
    got = run(dev(c))
    torch.cuda.synchronize()
    check(c, got)


def test_states_in_place():
    import momentum_delta_rule_gb300 as mdn
    for lens in ([90, 5], [2500]):
        c = case("bf16", lens, 1, 1, 64, 64, True)
        d = dev(c)
        want = run(d, train=False)
        S = d["S0"].clone()
        o, S_T = mdn.linear_attn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=d["scale"], S0=S, cu_seqlens=d["cu"], S_T=S)
        assert S_T is S and torch.equal(S, want["S_T"]) and torch.equal(o, want["o"])


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 70, 100], [0, 50, 70, 99], [0, -5, 70, 100], [0, 2000000000, 70, 100]])
def test_malformed_sequences_leave_outputs_alone(cu):
    import momentum_delta_rule_gb300 as mdn
    c = case("bf16", [40, 30, 30], 2, 1, 64, 64, True)
    d = dev(c)
    d["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    o = torch.full((1, 100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, S_T = mdn.linear_attn_fwd(d["q"], d["k"], d["v"], d["log_decay"], S0=d["S0"], cu_seqlens=d["cu"], o=o)
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert (o == 7).all() and torch.equal(S_T, d["S0"])
    g = mdn.linear_attn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], S0=d["S0"], dS_T=d["dS_T"], cu_seqlens=d["cu"])
    assert mdn.device_status() == mdn.MDN_ERR_INVALID_ARG
    assert torch.equal(g["dS0"], d["dS_T"])


def test_no_tokens():
    import momentum_delta_rule_gb300 as mdn
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    S0 = torch.randn(2, 3, 16, 8, device="cuda")
    args = (z(2, 0, 3, 16), z(2, 0, 3, 16), z(2, 0, 3, 8), torch.zeros(3, device="cuda"))
    o, S_T = mdn.linear_attn_fwd(*args, S0=S0)
    assert o.numel() == 0 and torch.equal(S_T, S0)
    g = mdn.linear_attn_bwd(*args, z(2, 0, 3, 8), dS_T=S0, need_dS0=True)
    assert torch.equal(g["dS0"], S0)
    assert mdn.linear_attn_fwd(*args)[1].abs().sum() == 0
    e = (z(0, 3, 16), z(0, 3, 16), z(0, 3, 8), torch.zeros(3, device="cuda"), torch.zeros(0, 3, 16, 8, device="cuda"))
    assert mdn.linear_attn_step(*e).shape == (0, 3, 8)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert torch.equal(mdn.linear_attn_fwd(z(1, 0, 3, 16), z(1, 0, 3, 16), z(1, 0, 3, 8), args[3], S0=S0, cu_seqlens=cu)[1], S0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,H,Hkv,dk,dv", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (5, 2, 2, 128, 128), (2, 3, 1, 57, 33),
                                           (2, 2, 2, 128, 20), (2, 1, 1, 100, 127), (4, 2, 1, 16, 32)])
def test_step(dtype, n, H, Hkv, dk, dv):
    import momentum_delta_rule_gb300 as mdn
    c = case(dtype, [1] * n, H, Hkv, dk, dv, packed=False, pad=3)
    d = dev(c)
    one = [d[x][:, 0] for x in ("q", "k", "v")]
    S_out = torch.empty_like(d["S0"])
    o = mdn.linear_attn_step(*one, d["log_decay"], d["S0"], scale=d["scale"], S_out=S_out)
    S = d["S0"].clone()
    o2 = mdn.linear_attn_step(*one, d["log_decay"], S, scale=d["scale"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S_out)
    # no operand of a step is rounded to bf16 but the result
    ref, mag = reference(c), reference(c, magnitude=True)
    for name, x, r, m in (("o", o, ref[0], mag[0]), ("S", S, ref[1], mag[1])):
        eps = torch.finfo(x.dtype).eps / 2
        off = np.abs(x.double().cpu().numpy().reshape(r.shape) - r)
        assert (off <= eps * np.abs(r) + (1 + eps) * (dk + 32) * 2.0 ** -24 * m + 1e-37).all(), name


def test_prompt_then_tokens():
    """Tokens one by one continue a prompt as the whole would."""
    import momentum_delta_rule_gb300 as mdn
    c = case("fp32", [140, 140], 2, 1, 64, 64, False)
    d = dev(c)
    cut = 129
    head = [d[x][:, :cut].contiguous() for x in ("q", "k", "v")]
    o, S = mdn.linear_attn_fwd(*head, d["log_decay"], scale=d["scale"], S0=d["S0"])
    outs = [o]
    for t in range(cut, 140):
        outs.append(mdn.linear_attn_step(*[d[x][:, t] for x in ("q", "k", "v")], d["log_decay"], S, scale=d["scale"])[:, None])
    torch.cuda.synchronize()
    check(c, dict(o=torch.cat(outs, 1), S_T=S))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nan_and_infinities_stay_with_their_sequence_and_run(dtype):
    """A bad token reaches its own run of 64 tokens, later ones of its sequence
    and the state, and nothing else."""
    for bad in (float("nan"), float("inf")):
        for name in ("q", "k", "v"):
            c = case(dtype, [200, 130], 2, 2, 64, 64, True)
            d = dev(c)
            want = run(d, train=False)
            d[name][0, 70, 0] = bad                   # sequence 0, its second run, head 0
            got = run(d, train=False)
            torch.cuda.synchronize()
            assert torch.equal(got["o"][:, :64], want["o"][:, :64])
            assert torch.equal(got["o"][:, 200:], want["o"][:, 200:])
            assert torch.equal(got["o"][:, :, 1], want["o"][:, :, 1])
            assert torch.equal(got["S_T"][1], want["S_T"][1]) and torch.equal(got["S_T"][0, 1], want["S_T"][0, 1])
            if name == "q":
                assert torch.equal(got["S_T"], want["S_T"])
                assert torch.equal(got["o"][:, 71:], want["o"][:, 71:]) and torch.equal(got["o"][:, :70], want["o"][:, :70])


def test_streams_devices_and_graphs():
    import momentum_delta_rule_gb300 as mdn
    c = case("bf16", [300, 80], 2, 1, 64, 64, True)
    d = dev(c)
    want = run(d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, S_T = mdn.linear_attn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=d["scale"], S0=d["S0"], cu_seqlens=d["cu"], stream=side)
    side.synchronize()
    assert torch.equal(o, want["o"]) and torch.equal(S_T, want["S_T"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(d)
    for t in got.values():
        t.zero_()
    d["v"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["o"], run(d)["o"])
    d["v"].div_(2)
    graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_workspace_of_the_caller():
    import momentum_delta_rule_gb300 as mdn
    c = case("bf16", [2100, 900], 2, 1, 32, 32, True)
    d = dev(c)
    want = run(d)
    sizes = (2, 3000, 2, 1, 32, 32, 1, mdn.MDN_BF16)
    fw, bw = (getattr(mdn.lib(), "mdn_linear_attn_%s_workspace_size" % x)(*sizes) for x in ("fwd", "bwd"))
    guard = 4096
    ws = torch.full((max(fw, bw) + guard,), 0x55, dtype=torch.uint8, device="cuda")
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    kw = dict(scale=d["scale"], S0=d["S0"], cu_seqlens=d["cu"])
    o, _ = mdn.linear_attn_fwd(*args, workspace=ws[:fw], **kw)
    assert (ws[fw:] == 0x55).all()
    g = mdn.linear_attn_bwd(*args, d["do"], dS_T=d["dS_T"], workspace=ws[:bw], **kw)
    assert (ws[bw:] == 0x55).all()
    assert torch.equal(o, want["o"]) and all(torch.equal(g[x], want[x]) for x in ("dq", "dk", "dv", "dS0"))
    with pytest.raises(mdn.MdnError):
        mdn.linear_attn_fwd(*args, workspace=ws[:256], **kw)


def test_rows_far_apart():
    """Token offsets beyond 2^31 elements."""
    import momentum_delta_rule_gb300 as mdn
    c = case("bf16", [130], 1, 1, 32, 32, True)
    d = dev(c)
    want = run(d)
    ld = (1 << 31) // 120 // 8 * 8
    base = torch.empty(130 * ld, dtype=torch.bfloat16, device="cuda")
    for name in ("q", "k", "v", "do"):
        far = torch.as_strided(base, (1, 130, 1, 32), (130 * ld, ld, 32, 1), {"q": 0, "k": 64, "v": 128, "do": 192}[name])
        far.copy_(d[name])
        d[name] = far
    got = run(d)
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_sequences(dtype):
    """More than a block orders by itself, some of them empty."""
    lens = [(7 * i) % 5 for i in range(700)]
    check_case(case(dtype, lens, 2, 1, 16, 24, True, seed=13))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_what_lies_behind_a_sequence_is_not_read(dtype):
    """Neighbours' rows come with a run's last tokens and are left out, whatever
    they hold."""
    c = case(dtype, [70, 58], 2, 2, 64, 64, True)
    d = dev(c)
    want = run(d)
    for name in ("q", "k", "v", "do"):
        d[name][0, 70:] = float("nan")
    got = run(d)
    torch.cuda.synchronize()
    for name in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[name][:, :70], want[name][:, :70]), name
    assert torch.equal(got["S_T"][0], want["S_T"][0]) and torch.equal(got["dS0"][0], want["dS0"][0])


def test_two_streams_at_once():
    import momentum_delta_rule_gb300 as mdn
    a, b = (dev(case(dt, [900, 33], 4, 2, 64, 64, True, seed=i)) for i, dt in enumerate(("bf16", "fp32")))
    want = [run(a), run(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, (d, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                got[i].append(run(d))
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    for w, gs in zip(want, got):
        for g in gs:
            for name in w:
                assert torch.equal(g[name], w[name]), name


def test_calls_one_behind_another():
    """Each call's kernels are set up while the one before it ends: what one call
    writes the next one reads whole."""
    import momentum_delta_rule_gb300 as mdn
    c = case("bf16", [1500, 1500], 2, 2, 64, 64, False)
    d = dev(c)
    args = (d["k"], d["v"], d["log_decay"])
    o, S = mdn.linear_attn_fwd(d["q"], *args, scale=d["scale"], S0=d["S0"])
    o2, S2 = mdn.linear_attn_fwd(o, *args, scale=d["scale"], S0=S)
    torch.cuda.synchronize()
    for _ in range(20):
        p, P = mdn.linear_attn_fwd(d["q"], *args, scale=d["scale"], S0=d["S0"])
        p2, P2 = mdn.linear_attn_fwd(p, *args, scale=d["scale"], S0=P)
        assert torch.equal(p2, o2) and torch.equal(P2, S2)


def test_outputs_of_any_alignment():
    import momentum_delta_rule_gb300 as mdn
    c = case("bf16", [100, 100], 2, 2, 64, 64, False)
    d = dev(c)
    want = run(d, train=False)["o"]
    buf = torch.zeros(want.numel() + 8, dtype=torch.bfloat16, device="cuda")
    for off in (1, 2, 3, 8):
        o = buf[off:off + want.numel()].view(want.shape)
        mdn.linear_attn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=d["scale"], S0=d["S0"], o=o)
        assert torch.equal(o, want)
        assert (buf[:off] == 0).all() and (buf[off + want.numel():] == 0).all()
        buf.zero_()
