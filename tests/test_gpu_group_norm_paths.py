"""The group norm on the GPU: calls and paths beside those of
test_gpu_group_norm.py (its tolerances)."""
import pytest
import torch

from tests.test_gpu_group_norm import case, check_case, dev, run

pytestmark = pytest.mark.gpu

MANY = [
    # more sequences than the gradient has clusters: packed ones that fit shared memory, and equal ones
    ([i % 3 for i in range(300)], 2048, 16, True),
    ([2] * 1000, 48, 3, False),
    # ... and than it has blocks for tiles, where the batch is too long for shared memory
    ([(7 * i) % 4 for i in range(4000)], 512, 1, True),
    ([0, 5000] + [1] * 700, 64, 4, True),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("lens,D,G,packed", MANY)
def test_more_sequences_than_sums(dtype, gate, lens, D, G, packed):
    check_case(case(dtype, lens, D, G, gate, over="sequence", packed=packed, seed=len(lens)))


@pytest.mark.parametrize("lens,D,G,packed", MANY)
def test_their_workspace_holds_what_is_written(lens, D, G, packed):
    import momentum_delta_rule_gb300 as mdn
    d = dev(case("bf16", lens, D, G, over="sequence", packed=packed))
    want = run(d)
    need = mdn.lib().mdn_group_norm_bwd_workspace_size(len(lens), sum(lens), D, G, 1, mdn.MDN_BF16)
    ws = torch.full((need + 4096,), 0x55, dtype=torch.uint8, device="cuda")
    g = mdn.group_norm_bwd(d["x"], G, want["stats"], d["dy"], weight=d["weight"], bias=d["bias"], gate=d["gate"], activation="silu",
                           over="sequence", cu_seqlens=d["cu"], workspace=ws[:need])
    assert all(torch.equal(g[n], want[n]) for n in g)
    assert (ws[need:] == 0x55).all()


@pytest.mark.parametrize("over,D,G", [("token", 32, 2), ("token", 4096, 1), ("sequence", 32, 2), ("sequence", 4096, 1)])
def test_rows_far_apart(over, D, G):
    """Token offsets beyond 2^31 elements."""
    d = dev(case("bf16", [100, 30], D, G, over=over))
    want = run(d)
    ld = (1 << 31) // 120 // 8 * 8
    base = torch.empty(130 * ld, dtype=torch.bfloat16, device="cuda")
    for i, name in enumerate(("x", "gate", "dy")):
        far = torch.as_strided(base, (1, 130, D), (130 * ld, ld, 1), i * D)
        far.copy_(d[name])
        d[name] = far
    got = run(d)
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_two_streams_at_once():
    import momentum_delta_rule_gb300 as mdn
    cases = [dev(case("bf16", [900, 33], 128, 4, over="sequence")), dev(case("fp32", [700], 96, 3)),
             dev(case("fp32", [9000], 64, 1, over="sequence", seed=1))]
    want = [run(d) for d in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(10):
        for i, (d, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(run_alone(d))
    torch.cuda.synchronize()
    assert mdn.device_status() == mdn.MDN_OK
    for w, gs in zip(want, got):
        for g in gs:
            for name in w:
                assert torch.equal(g[name], w[name]), name


def run_alone(d):
    """`run` without a comparison, which would wait."""
    import momentum_delta_rule_gb300 as mdn
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], activation=d["activation"], over=d["over"], center=d["center"],
              cu_seqlens=d["cu"])
    y, stats = mdn.group_norm_fwd(d["x"], d["groups"], return_stats=True, **kw)
    return dict(y=y, stats=stats, **mdn.group_norm_bwd(d["x"], d["groups"], stats, d["dy"], **kw))


@pytest.mark.parametrize("over,lens,D,G", [("token", [3000], 64, 4), ("token", [700], 4608, 1), ("sequence", [300, 200], 96, 3),
                                           ("sequence", [9000], 64, 1)])
def test_calls_one_behind_another(over, lens, D, G):
    """A call's kernels are set up while those before them end: what one writes the
    next one reads whole."""
    import momentum_delta_rule_gb300 as mdn
    d = dev(case("bf16", lens, D, G, over=over))
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], activation="silu", over=over, cu_seqlens=d["cu"])

    def chain():
        y, stats = mdn.group_norm_fwd(d["x"], G, return_stats=True, **kw)
        g = mdn.group_norm_bwd(d["x"], G, stats, y, **kw)
        h = mdn.group_norm_bwd(d["x"], G, stats, g["dx"], **kw)
        return mdn.group_norm_fwd(h["dx"], G, **kw), h["dw"], h["dbias"]

    want = chain()
    torch.cuda.synchronize()
    for _ in range(20):
        for a, b in zip(chain(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("over,lens", [("token", [40, 30]), ("sequence", [40, 30]), ("sequence", [40, 6000])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["x", "gate", "dy"])
def test_a_bad_value_stays_in_its_group_in_the_gradient(over, lens, bad, name):
    d = dev(case("fp32", lens, 64, 4, over=over))
    want = run_alone(d)
    d[name][0, 10, 20] = bad                     # group 1: columns 16 to 31
    got = run_alone(d)
    rows = slice(10, 11) if over == "token" else slice(0, lens[0])
    for g in ("dx", "dgate"):
        assert not got[g][0, 10, 16:32].isfinite().all()
        got[g][0, rows, 16:32] = want[g][0, rows, 16:32]
        assert torch.equal(got[g], want[g]), g
    for g in ("dw", "dbias"):
        got[g][16:32] = want[g][16:32]
        assert torch.equal(got[g], want[g]), g
