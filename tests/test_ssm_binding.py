"""The state-space binding's handling of streams, and the example's of
states (no GPU needed)."""
import importlib.util
import os
import types

import pytest
import torch

from momentum_delta_rule_gb300 import ssm


def test_a_stream_of_another_device_is_refused():
    # the call would switch back to the tensors' device, and to its current stream
    t = types.SimpleNamespace(device=torch.device("cuda", 0))
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        ssm._on(t, other)


def _example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("selective_layer",
                                                  os.path.join(root, "examples", "selective_layer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def test_the_example_fills_an_empty_state(monkeypatch):
    # a prompt from scratch: the caller's dict is empty until the prompt has run
    ex, seen = _example(), {}

    def conv(x, w, bias=None, state=None, cu_seqlens=None, output_final_state=False):
        seen.update(conv=state)
        return x, "conv" if output_final_state else None

    def scan(u, *args, h0=None, output_final_state=True, **kw):
        seen.update(ssm=h0)
        return u, "ssm" if output_final_state else None

    monkeypatch.setattr(ex.mdn, "short_conv_fwd", conv)
    monkeypatch.setattr(ex.mdn, "ssm_scan_fwd", scan)
    monkeypatch.setattr(ex.mdn, "norm_residual_fwd", lambda y, x, **kw: (x, y))
    layer = ex.Layer(16, 32, dtype=torch.float32, device="cpu")
    x, state = torch.zeros(1, 3, 16), {}
    layer.prompt(x, x, state=state)
    assert seen == dict(conv=None, ssm=None) and state == dict(conv="conv", ssm="ssm")
    layer.prompt(x, x, state=state)                 # and goes on from there
    assert seen == dict(conv="conv", ssm="ssm")
    layer.prompt(x, x)
    assert seen == dict(conv=None, ssm=None)


def test_the_example_differentiates_a_prompt_that_goes_on(monkeypatch):
    # the convolution's gradient needs the tokens before the prompt, as its forward had them
    ex, seen = _example(), {}
    x, stats = torch.zeros(1, 3, 16), torch.zeros(1, 3, 2)
    tokens = lambda u, **kw: (u, torch.ones(1), torch.ones(1))
    monkeypatch.setattr(ex.mdn, "short_conv_fwd", lambda x, w, **kw: (x, torch.ones(1, 3, 32)))
    monkeypatch.setattr(ex.mdn, "ssm_scan_fwd", lambda u, *a, **kw: tokens(u))
    monkeypatch.setattr(ex.mdn, "norm_residual_fwd", lambda y, x, **kw: (x, y, stats))
    monkeypatch.setattr(ex.mdn, "norm_residual_bwd", lambda y, x, *a, **kw: dict.fromkeys(
        ("dy", "dx", "dw_post", "dw_pre", "dscale"), y))
    monkeypatch.setattr(ex.mdn, "ssm_scan_bwd", lambda u, dt, A, Bm, Cm, *a, **kw: dict(
        du=u, ddt=dt, dz=u, dA=A, dB=Bm, dC=Cm, dD_skip=A, ddt_bias=A))
    monkeypatch.setattr(ex.mdn, "short_conv_bwd", lambda x, w, dy, state=None, **kw: seen.update(state=state) or dict(
        dx=x, dw=w, dbias=w))
    layer = ex.Layer(16, 32, dtype=torch.float32, device="cpu")
    before = torch.full((1, 3, 32), 2.0)
    for state in (None, {}, {"conv": before, "ssm": None}):
        save, given = {}, None if not state else before
        layer.prompt(x, x, state=state, save=save)
        layer.gradient(save, x, x)
        assert seen["state"] is given
