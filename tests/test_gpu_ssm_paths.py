"""GPU parity of the state-space layer's operators on the paths that whole
prompts and training batches take: convolution runs of many batches of rows,
gradient blocks that go through several items, sequences cut into segments.
``tests/test_ssm_launches.py`` checks without a GPU that these sizes do so.

Tolerances are those of ``tests/test_gpu_ssm.py``, and where it is said a bound
on the relative L2 error of an fp32 output: an elementwise bound has to allow
every rounding of a long sequence in the same direction, about 2^-24 a token,
while the errors of a sum average out.  A state remembers some tens of tokens
here, and a token's step is off by a few 2^-24 and the exponential's 2^-22:
about 1e-6 together, and 1e-5 leaves room for the sums over tokens.
"""
import threading

import pytest
import torch

from tests.test_gpu_ssm import TD, _dev, _gen, _np, _scan_kw, _scan_ref, check_conv, check_scan, conv_case, scan_case

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- convolution

# (dtype, D, tokens): packets of four channels, of two, and single ones
CONV_RUNS = [("bf16", 8192, 2003), ("bf16", 8190, 1203), ("bf16", 8191, 603), ("bf16", 2047, 2403),
             ("fp32", 8192, 2003), ("fp32", 8191, 603), ("bf16", 2048, 8011)]


def ragged(tokens, seed):
    """Short sequences that end on, before and behind the batches' boundaries,
    empty ones among them, then long ones."""
    g = torch.Generator().manual_seed(seed)
    lens = [8, 8, 7, 1, 9, 0, 3, 4, 4, 0, 0, 16, 15, 17, 12]
    while sum(lens) < tokens // 2:
        lens.append(int(torch.randint(0, 25, (1,), generator=g)))
    rest = tokens - sum(lens)
    return lens + [rest // 3, rest - rest // 3, 0]


@pytest.mark.parametrize("dtype,D,tokens", CONV_RUNS)
@pytest.mark.parametrize("W", [2, 4])
def test_conv_runs_of_many_batches(dtype, D, tokens, W):
    check_conv(conv_case(dtype, ragged(tokens, D + W), D=D, W=W, strided=D % 2 == 0, seed=W))


@pytest.mark.parametrize("dtype,D,tokens", [("bf16", 8192, 2004), ("bf16", 8191, 604), ("fp32", 8192, 2004)])
def test_conv_runs_of_many_batches_equal_lengths(dtype, D, tokens):
    check_conv(conv_case(dtype, [tokens // 4] * 4, D=D, W=3, packed=False, strided=False, seed=3), silu=False)


# ---------------------------------------------------------- scan's gradient

# (dtype, lens, D, N, G, packed): more items than blocks share them
MANY_ITEMS = [
    ("bf16", [40, 33, 32, 31, 64, 1, 0, 47, 50, 5, 38, 61, 2, 36, 70], 4096, 16, 1, True),
    ("fp32", [40, 33, 32, 31, 64, 1, 0, 47, 50, 5, 38, 61, 2, 36, 70], 4096, 16, 2, True),
    ("bf16", [37] * 14, 4096, 16, 1, False),
    ("bf16", [20, 41, 33, 1, 0, 35, 64, 7, 29, 40, 32, 18, 34], 1024, 33, 1, True),
    ("fp32", [150] * 3, 2048, 33, 1, False),
    ("fp32", [9, 65, 30, 1, 33, 0, 12, 40, 34, 8, 31, 35], 512, 128, 2, True),
]


@pytest.mark.parametrize("case", MANY_ITEMS, ids=lambda c: "%s-%d-%d-%s" % (c[0], c[2], c[3], "packed" if c[5] else "equal"))
def test_scan_gradient_of_several_items_a_block(case):
    dtype, lens, D, N, G, packed = case
    check_scan(scan_case(dtype, lens, D=D, N=N, G=G, packed=packed, seed=N), train=True)


# --------------------------------------------------- relative errors, fp32

CUT = [([3000], 64, 16, False), ([1500, 1500], 66, 16, False), ([2600, 40, 900], 48, 8, True), ([1200], 16, 64, False)]


@pytest.mark.parametrize("lens,D,N,packed", CUT)
def test_scan_errors_of_cut_sequences(lens, D, N, packed):
    import momentum_delta_rule_gb300 as mdn
    c = scan_case("fp32", lens, D=D, N=N, packed=packed, seed=N)
    d = _dev(c)
    args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"])
    y, hT, hc = mdn.ssm_scan_fwd(*args, h0=d["h0"], return_chunk_states=True, **_scan_kw(d))
    dy, dhT = torch.randn(y.shape, generator=_gen(5)), torch.randn(hT.shape, generator=_gen(6))
    g = mdn.ssm_scan_bwd(*args, hc, dy.cuda(), dh_T=dhT.cuda(), need_dh0=True, **_scan_kw(d))
    ref = _scan_ref(c, dy=_np(dy).reshape(-1, D), dh_T=_np(dhT))
    got = dict(g, y=y, h_T=hT)
    for k, want in dict(ref[3], y=ref[0], h_T=ref[1]).items():
        want = torch.from_numpy(want)
        err = float((got[k].double().cpu().reshape(want.shape) - want).norm() / want.norm())
        assert err <= 1e-5, (k, err)


# ------------------------------------------------------------ host threads

def test_norms_of_two_widths_from_two_threads():
    import momentum_delta_rule_gb300 as mdn

    def case(dtype, D):
        g = _gen(D)
        y, x, dX, dh = (torch.randn(300, D, generator=g).to(TD[dtype]).cuda() for _ in range(4))
        w = torch.randn(D, generator=g).cuda()
        return dtype, y, x, w, dX, dh

    def run(c):
        _, y, x, w, dX, dh = c
        X, h, st = mdn.norm_residual_fwd(y, x, w_post=w, w_pre=w, return_stats=True)
        g = mdn.norm_residual_bwd(y, x, st, dX, dh=dh, w_post=w, w_pre=w)
        return [X, h, g["dy"], g["dx"], g["dw_post"], g["dw_pre"]]

    # widths that share a kernel: 4096 and 8192 of the forward, 2048 and 4096 of the gradient
    cases = [case("bf16", 4096), case("bf16", 8192), case("fp32", 2048), case("fp32", 4096)]
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    failures = []

    def work(mine):
        try:
            for _ in range(150):
                for c, _ in mine:
                    run(c)
            torch.cuda.synchronize()
            for c, w in mine:
                if not all(torch.equal(a, b) for a, b in zip(run(c), w)):
                    failures.append("results differ")
        except Exception as e:                      # reported by the main thread
            failures.append(repr(e))

    pairs = list(zip(cases, want))
    threads = [threading.Thread(target=work, args=(m,)) for m in (pairs[::2], pairs[1::2])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
