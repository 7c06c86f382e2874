"""Linear attention on the GPU: calls and paths beside those of test_gpu_attn.py
(its tolerances)."""
import pytest
import torch

from tests.test_gpu_attn import case, check_case, dev, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", [0, 1])
def test_without_tokens_nothing_but_the_states_is_needed(code):
    import momentum_delta_rule_gb300 as mdn
    L = mdn.lib()
    S0, out = torch.randn(2, 3, 16, 8, device="cuda"), torch.empty(2, 3, 16, 8, device="cuda")

    def fwd(S0, S_T, handle):
        return L.mdn_linear_attn_fwd(None, None, None, None, S0, None, S_T, None, 2, 2, 0, 3, 3, 16, 8, 1.0, 48, 48, 24, code, None, 0, handle)

    def bwd(dS_T, dS0, handle):
        return L.mdn_linear_attn_bwd(None, None, None, None, None, None, dS_T, None, None, None, dS0, None, 2, 2, 0, 3, 3, 16, 8, 1.0,
                                     48, 48, 24, 24, code, None, 0, handle)

    for call in (fwd, bwd):
        stream = torch.cuda.current_stream()
        for given, want in ((S0, S0), (None, torch.zeros_like(S0))):
            out.fill_(7)
            assert call(None if given is None else given.data_ptr(), out.data_ptr(), stream.cuda_stream) == 0
            assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            assert call(S0.data_ptr(), out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, S0)
    assert fwd(S0.data_ptr(), S0.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert mdn.device_status() == mdn.MDN_OK


# Cut sequences whose segments each join the states of those before them (few
# segments), in the directions and types named: partial last segments, an empty
# sequence, shared heads, widths that differ.
JOINED = [
    # lens, H, Hkv, dk, dv, packed, where
    ([960, 960], 24, 24, 32, 32, False, ("fwd fp32", "fwd bf16")),
    ([950, 930], 24, 12, 40, 24, True, ("fwd fp32", "fwd bf16")),
    ([310, 330], 16, 8, 32, 16, True, ("fwd fp32",)),
    ([950] * 4, 4, 2, 40, 24, False, ("bwd fp32", "bwd bf16")),
    ([950, 930, 970, 960], 4, 2, 32, 48, True, ("bwd fp32", "bwd bf16")),
    ([950, 0, 990, 960], 4, 2, 32, 48, True, ("bwd fp32",)),
    ([320] * 3, 4, 1, 64, 128, False, ("bwd fp32",)),
]
# Cut sequences whose states a kernel joins, elements one at a time (odd sizes)
# and four, with rows that move one element, two and sixteen bytes at a time.
COMBINED = [
    # lens, H, Hkv, dk, dv, packed, offset
    ([2500], 2, 1, 57, 33, False, 0),
    ([1100, 3, 0, 3300], 2, 2, 127, 1, True, 0),
    ([2500], 2, 1, 58, 34, False, 0),
    ([2500], 2, 2, 64, 64, False, 1),
    ([1100, 3, 0, 3300], 2, 2, 64, 64, True, 2),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed,where", JOINED)
def test_segments_that_join_the_states_before_them(dtype, lens, H, Hkv, dk, dv, packed, where):
    check_case(case(dtype, lens, H, Hkv, dk, dv, packed, seed=31))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,H,Hkv,dk,dv,packed,offset", COMBINED)
def test_segments_whose_states_a_kernel_joins(dtype, lens, H, Hkv, dk, dv, packed, offset):
    check_case(case(dtype, lens, H, Hkv, dk, dv, packed, offset=offset, seed=37))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("i", [0, 1])
def test_joining_segments_with_states_in_place(dtype, i):
    import momentum_delta_rule_gb300 as mdn
    lens, H, Hkv, dk, dv, packed, _ = JOINED[i]
    d = dev(case(dtype, lens, H, Hkv, dk, dv, packed, seed=41))
    want = run(d, train=False)
    for _ in range(5):
        S = d["S0"].clone()
        o, S_T = mdn.linear_attn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=d["scale"], S0=S, cu_seqlens=d["cu"], S_T=S)
        assert S_T is S and torch.equal(S, want["S_T"]) and torch.equal(o, want["o"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_a_bad_token_does_not_reach_in_the_gradient(dtype, bad):
    """dq takes v and k of earlier tokens and the run's own, dk and dv q and do of
    later ones and the run's own; a gradient does not take the row that it belongs
    to."""
    c = case(dtype, [200, 130], 2, 2, 64, 64, True)
    want = run(dev(c))
    same = {  # tokens of sequence 0, head 0 that the bad row 70 does not reach
        "q": dict(dq=slice(0, 200), dk=slice(128, 200), dv=slice(128, 200)),
        "k": dict(dq=slice(0, 64), dk=slice(0, 200), dv=[t for t in range(200) if t != 70]),
        "v": dict(dq=slice(0, 64), dk=[t for t in range(200) if t != 70], dv=slice(0, 200)),
        "do": dict(dq=[t for t in range(200) if t != 70], dk=slice(128, 200), dv=slice(128, 200)),
    }
    for name, tokens in same.items():
        d = dev(c)
        d[name][0, 70, 0] = bad
        got = run(d)
        torch.cuda.synchronize()
        for g, t in tokens.items():
            assert torch.equal(got[g][0, t, 0], want[g][0, t, 0]), (name, g)
            assert torch.equal(got[g][:, :, 1], want[g][:, :, 1]), (name, g)
            assert torch.equal(got[g][:, 200:], want[g][:, 200:]), (name, g)
        assert torch.equal(got["dS0"][1], want["dS0"][1]) and torch.equal(got["dS0"][0, 1], want["dS0"][0, 1])
        if name in ("k", "v"):
            assert torch.equal(got["dS0"], want["dS0"])
