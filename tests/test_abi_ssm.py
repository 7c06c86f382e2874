"""Refusals of the state-space layer's entry points and the host-side rules of
their binding (no GPU needed: validation runs before any device work)."""
import ctypes

import pytest
import torch

import momentum_delta_rule_gb300 as mdn
from momentum_delta_rule_gb300 import ssm


@pytest.fixture(scope="module")
def L():
    from momentum_delta_rule_gb300 import build
    build.build()
    return mdn.lib()


P = lambda a: ctypes.c_void_p(a)          # addresses that are never dereferenced


def _call(fn, defaults, over):
    args = dict(defaults)
    for k in over:
        assert k in args, k
    args.update(over)
    return fn(*args.values())


CONV = dict(x=P(0x1000), w=P(0x2000), bias=None, s0=None, y=P(0x3000), sT=None, cu=None, n_seq=2, B=2, T=8, D=16,
            W=4, act=1, ld=16, dtype=1, stream=None)
CONV_BWD = dict(x=P(0x1000), w=P(0x2000), bias=None, s0=None, dy=P(0x3000), dsT=None, dx=P(0x4000), dw=P(0x5000),
                db=None, ds0=None, cu=None, n_seq=2, B=2, T=8, D=16, W=4, act=1, ld=16, ld_dy=16, dtype=1,
                ws=P(0x10000), bytes=1 << 30, stream=None)
CONV_STEP = dict(x=P(0x1000), w=P(0x2000), bias=None, s=P(0x3000), so=P(0x3000), y=P(0x4000), N=4, D=16, W=4, act=1,
                 ld=16, dtype=1, stream=None)
SCAN = dict(u=P(0x1000), dt=P(0x2000), A=P(0x3000), B=P(0x4000), C=P(0x5000), D_skip=None, z=None, bias=None,
            h0=None, y=P(0x6000), hT=None, hc=None, cu=None, n_seq=2, Bn=2, T=8, D=16, G=2, N=16, softplus=1, ld_u=16,
            ld_dt=16, ld_B=32, ld_C=32, ld_z=16, dtype=1, ws=P(0x10000), bytes=1 << 30, stream=None)
SCAN_BWD = dict(u=P(0x1000), dt=P(0x2000), A=P(0x3000), B=P(0x4000), C=P(0x5000), D_skip=None, z=None, bias=None,
                hc=P(0x6000), dy=P(0x7000), dhT=None, du=P(0x8000), ddt=P(0x9000), dA=P(0xa000), dB=P(0xb000),
                dC=P(0xc000), dD=None, dz=None, dbias=None, dh0=None, cu=None, n_seq=2, Bn=2, T=8, D=16, G=2, N=16,
                softplus=1, ld_u=16, ld_dt=16, ld_B=32, ld_C=32, ld_z=16, ld_dy=16, dtype=1, ws=P(0x10000),
                bytes=1 << 30, stream=None)
SCAN_STEP = dict(u=P(0x1000), dt=P(0x2000), A=P(0x3000), B=P(0x4000), C=P(0x5000), D_skip=None, z=None, bias=None,
                 h=P(0x6000), ho=P(0x6000), y=P(0x7000), n=4, D=16, G=2, N=16, softplus=1, ld_u=16, ld_dt=16, ld_B=32,
                 ld_C=32, ld_z=16, dtype=1, stream=None)
NORM = dict(y=P(0x1000), x=P(0x2000), gate=None, w1=None, w2=None, scale=None, xo=P(0x3000), h=None, stats=None,
            rows=4, D=16, act=0, eps=1e-6, ld_y=16, ld_x=16, ld_g=16, dtype=1, stream=None)
NORM_BWD = dict(y=P(0x1000), x=P(0x2000), gate=None, w1=None, w2=None, scale=None, stats=P(0x3000), dxo=P(0x4000),
                dh=None, dy=P(0x5000), dx=P(0x6000), dgate=None, dw1=None, dw2=None, dsc=None, rows=4, D=16, act=0,
                ld_y=16, ld_x=16, ld_g=16, ld_dxo=16, ld_dh=16, dtype=1, ws=P(0x10000), bytes=1 << 30, stream=None)

# what every call with sequences refuses
BATCH = [(dict(n_seq=3), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(dtype=5), 1), (dict(cu=P(0x7000)), 1),
         (dict(cu=P(0x7002), n_seq=1), 1), (dict(T=1 << 30), 1)]


@pytest.mark.parametrize("over,code", BATCH + [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(y=P(0x1000)), 1), (dict(ld=15), 1),
    (dict(x=P(0x1001)), 1), (dict(w=P(0x2002)), 1), (dict(act=2), 1), (dict(s0=P(0x8000), sT=P(0x8000)), 1),
    (dict(W=1), 2), (dict(W=5), 2),
])
def test_short_conv_fwd_rejects(L, over, code):
    assert _call(L.mdn_short_conv_fwd, CONV, over) == code


@pytest.mark.parametrize("over,code", BATCH + [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(dx=P(0x3000)), 1), (dict(ld_dy=15), 1),
    (dict(ws=None), 1), (dict(bytes=16), 1), (dict(ws=P(0x10010)), 1), (dict(db=P(0x5000)), 1), (dict(W=5), 2),
])
def test_short_conv_bwd_rejects(L, over, code):
    assert _call(L.mdn_short_conv_bwd, CONV_BWD, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(x=None), 1), (dict(s=None), 1), (dict(so=None), 1), (dict(y=P(0x3000)), 1), (dict(N=-1), 1), (dict(ld=8), 1),
    (dict(so=P(0x1000)), 1), (dict(W=5), 2),
])
def test_short_conv_step_rejects(L, over, code):
    assert _call(L.mdn_short_conv_step, CONV_STEP, over) == code


SCAN_COMMON = [(dict(u=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(C=None), 1),
               (dict(G=3), 1), (dict(G=0), 1), (dict(N=0), 1), (dict(ld_u=15), 1), (dict(ld_dt=15), 1),
               (dict(ld_B=31), 1), (dict(ld_C=31), 1), (dict(z=P(0xe000), ld_z=15), 1), (dict(A=P(0x3002)), 1),
               (dict(N=129, ld_B=258, ld_C=258), 2)]


@pytest.mark.parametrize("over,code", BATCH + SCAN_COMMON + [
    (dict(y=None), 1), (dict(y=P(0x1000)), 1), (dict(hT=P(0x6000)), 1), (dict(h0=P(0x8004)), 1),
    (dict(hc=P(0x8008)), 1), (dict(hT=P(0x8000), hc=P(0x8000)), 1), (dict(cu=P(0x7000), n_seq=4, Bn=1, ws=None), 1),
    (dict(cu=P(0x7000), n_seq=4, Bn=1, bytes=8), 1),
])
def test_ssm_scan_fwd_rejects(L, over, code):
    assert _call(L.mdn_ssm_scan_fwd, SCAN, over) == code


@pytest.mark.parametrize("over,code", BATCH + SCAN_COMMON + [
    (dict(hc=None), 1), (dict(dy=None), 1), (dict(du=None), 1), (dict(dA=None), 1), (dict(dB=None), 1),
    (dict(dC=P(0xb000)), 1), (dict(du=P(0x1000)), 1), (dict(z=P(0xe000)), 1), (dict(ld_dy=15), 1), (dict(ws=None), 1),
    (dict(bytes=256), 1), (dict(ws=P(0x10008)), 1), (dict(dh0=P(0xe004)), 1),
])
def test_ssm_scan_bwd_rejects(L, over, code):
    assert _call(L.mdn_ssm_scan_bwd, SCAN_BWD, over) == code


@pytest.mark.parametrize("over,code", SCAN_COMMON + [
    (dict(h=None), 1), (dict(ho=None), 1), (dict(y=None), 1), (dict(n=-1), 1), (dict(y=P(0x6000)), 1),
    (dict(ho=P(0x3000)), 1), (dict(h=P(0x6004)), 1),
])
def test_ssm_scan_step_rejects(L, over, code):
    assert _call(L.mdn_ssm_scan_step, SCAN_STEP, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(y=None), 1), (dict(x=None), 1), (dict(xo=None), 1), (dict(w2=P(0x8000)), 1), (dict(xo=P(0x1000)), 1),
    (dict(ld_x=24, xo=P(0x2000)), 1), (dict(rows=-1), 1), (dict(D=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(act=2), 1), (dict(gate=P(0x9000), ld_g=8), 1), (dict(stats=P(0x9004)), 1),
    (dict(D=16385, ld_y=16385, ld_x=16385), 2),
])
def test_norm_residual_fwd_rejects(L, over, code):
    assert _call(L.mdn_norm_residual_fwd, NORM, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(stats=None), 1), (dict(dxo=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dy=P(0x1000)), 1),
    (dict(gate=P(0x9000)), 1), (dict(w1=P(0x9000)), 1), (dict(w2=P(0x9000), dw2=P(0xa000)), 1),
    (dict(scale=P(0x9000)), 1), (dict(ld_dxo=24, dx=P(0x4000)), 1), (dict(ws=None), 1), (dict(bytes=8), 1),
    (dict(D=16385, ld_y=16385, ld_x=16385, ld_dxo=16385), 2),
])
def test_norm_residual_bwd_rejects(L, over, code):
    assert _call(L.mdn_norm_residual_bwd, NORM_BWD, over) == code


def test_sizes(L):
    assert mdn.ssm_state_slots(2, 2, 33, False) == 4
    assert mdn.ssm_state_slots(3, 1, 100, True) == 100 // 32 + 3
    assert mdn.ssm_state_slots(0, 0, 0, False) == 0 and mdn.ssm_state_slots(-1, 1, 5, True) == 0
    for f in (L.mdn_ssm_scan_fwd_workspace_size, L.mdn_ssm_scan_bwd_workspace_size):
        assert f(4, 100, 64, 2, 16, 1) % 256 == 0 and f(4, 100, 64, 2, 16, 1) > 0
        assert f(4, 100, 64, 3, 16, 1) == 0 and f(4, 100, 64, 2, 129, 1) == 0 and f(-1, 100, 64, 2, 16, 1) == 0
    assert L.mdn_short_conv_bwd_workspace_size(100, 64, 4, 1) > 0
    assert L.mdn_short_conv_bwd_workspace_size(100, 64, 5, 1) == 0
    assert L.mdn_norm_residual_bwd_workspace_size(100, 64, 0) > 0
    assert L.mdn_norm_residual_bwd_workspace_size(100, 16385, 0) == 0


def test_row_strides():
    x = torch.zeros(2, 5, 24)
    assert ssm._row_stride("x", x, 1) == 24
    assert ssm._row_stride("x", x[..., :8], 1) == 24
    assert ssm._row_stride("x", x[:, :1, :8], 1) == 120          # one token a sequence
    assert ssm._row_stride("x", x[:1, :, 8:], 1) == 24
    assert ssm._row_stride("x", x[..., :12].unflatten(-1, (3, 4)), 2) == 24
    assert ssm._row_stride("x", x[:, :0], 1) == 24
    for bad in (x[:, :3], x[..., ::2], x.transpose(1, 2), x[:1, :1].expand(2, 5, 24)):
        with pytest.raises(ValueError):
            ssm._row_stride("x", bad, 1)
    with pytest.raises(ValueError):
        ssm._row_stride("x", x[..., :16].unflatten(-1, (4, 4))[..., :3], 2)


def test_binding_refuses_cpu_tensors_and_bad_names():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        mdn.short_conv_fwd(x, w)
    with pytest.raises(ValueError):
        mdn.ssm_scan_fwd(x, x, torch.zeros(8, 2), x.unflatten(-1, (4, 2)), x.unflatten(-1, (4, 2)))
    with pytest.raises(ValueError):
        mdn.norm_residual_fwd(x, x)
    with pytest.raises(TypeError):
        mdn.short_conv_fwd(x.half(), w)
    with pytest.raises(ValueError):
        ssm._act(ssm._CONV_ACT, "activation", "gelu")
