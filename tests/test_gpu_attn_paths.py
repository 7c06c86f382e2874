"""Linear attention on the GPU: calls and paths beside those of test_gpu_attn.py
(its tolerances)."""
import pytest
import torch

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
