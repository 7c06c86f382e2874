"""Refusals of linear attention's and the group norm's entry points and the
host-side rules of their binding (no GPU needed: validation runs before any
device work)."""
import ctypes

import pytest
import torch

import momentum_delta_rule_gb300 as mdn
from tests.test_abi_ssm import P, _call


@pytest.fixture(scope="module")
def L():
    from momentum_delta_rule_gb300 import build
    build.build()
    return mdn.lib()


FWD = dict(q=P(0x1000), k=P(0x2000), v=P(0x3000), log_decay=P(0x4000), S0=None, o=P(0x5000), S_T=None, cu=None, n_seq=2,
           B=2, T=8, H=4, Hkv=2, dk=16, dv=8, scale=1.0, ld_q=64, ld_k=32, ld_v=16, dtype=1, ws=P(0x10000), bytes=1 << 40,
           stream=None)
BWD = dict(q=P(0x1000), k=P(0x2000), v=P(0x3000), log_decay=P(0x4000), S0=None, do=P(0x5000), dS_T=None, dq=P(0x6000),
           dk_out=P(0x7000), dv_out=P(0x8000), dS0=None, cu=None, n_seq=2, B=2, T=8, H=4, Hkv=2, dk=16, dv=8, scale=1.0,
           ld_q=64, ld_k=32, ld_v=16, ld_do=32, dtype=1, ws=P(0x10000), bytes=1 << 40, stream=None)
STEP = dict(q=P(0x1000), k=P(0x2000), v=P(0x3000), log_decay=P(0x4000), S=P(0x5000), S_out=P(0x5000), o=P(0x6000), n=4, H=4,
            Hkv=2, dk=16, dv=8, scale=1.0, ld_q=64, ld_k=32, ld_v=16, dtype=1, stream=None)
GN = dict(x=P(0x1000), gate=None, w=None, b=None, y=P(0x2000), stats=None, cu=None, n_seq=2, B=2, T=8, D=16, G=4, over=1,
          center=1, act=1, eps=1e-5, ld_x=16, ld_g=16, dtype=1, ws=P(0x10000), bytes=1 << 40, stream=None)
GN_BWD = dict(x=P(0x1000), gate=None, w=None, b=None, stats=P(0x2000), dy=P(0x3000), dx=P(0x4000), dgate=None, dw=None,
              db=None, cu=None, n_seq=2, B=2, T=8, D=16, G=4, over=1, center=1, act=1, ld_x=16, ld_g=16, ld_dy=16, dtype=1,
              ws=P(0x10000), bytes=1 << 40, stream=None)

HEADS = [(dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(log_decay=None), 1), (dict(H=3), 1), (dict(H=0), 1),
         (dict(Hkv=0), 1), (dict(dk=0), 1), (dict(dv=0), 1), (dict(ld_q=63), 1), (dict(ld_k=31), 1), (dict(ld_v=15), 1),
         (dict(dtype=2), 1), (dict(q=P(0x1001)), 1), (dict(log_decay=P(0x4002)), 1),
         (dict(dk=129, ld_q=516, ld_k=258), 2), (dict(dv=129, ld_v=258, ld_do=516), 2)]
BATCH = [(dict(n_seq=3), 1), (dict(T=-1), 1), (dict(cu=P(0x9000)), 1), (dict(cu=P(0x9002), n_seq=1), 1), (dict(T=1 << 30), 1),
         (dict(B=0, n_seq=0, T=-3), 1)]


def _only(d, over):
    return {k: v for k, v in over.items() if k in d}


@pytest.mark.parametrize("over,code", HEADS + BATCH + [
    (dict(o=None), 1), (dict(o=P(0x1000)), 1), (dict(S0=P(0xa000), S_T=P(0xb004)), 1), (dict(S0=P(0xa004)), 1),
    (dict(S_T=P(0x5000)), 1), (dict(cu=P(0x9000), B=1, ws=None), 1), (dict(cu=P(0x9000), B=1, bytes=16), 1),
    (dict(cu=P(0x9000), B=1, ws=P(0x10010)), 1), (dict(B=1, n_seq=1, T=20000, ws=None), 1)])
def test_linear_attn_fwd_rejects(L, over, code):
    assert _call(L.mdn_linear_attn_fwd, FWD, _only(FWD, over)) == code


@pytest.mark.parametrize("over,code", HEADS + BATCH + [
    (dict(do=None), 1), (dict(dq=None), 1), (dict(dk_out=None), 1), (dict(dv_out=None), 1), (dict(dq=P(0x1000)), 1),
    (dict(dk_out=P(0x6000)), 1), (dict(ld_do=31), 1), (dict(dS0=P(0xa004)), 1), (dict(dS_T=P(0xa000), dS0=P(0xa000)), 1),
    (dict(ws=None), 1), (dict(bytes=16), 1), (dict(ws=P(0x10008)), 1)])
def test_linear_attn_bwd_rejects(L, over, code):
    assert _call(L.mdn_linear_attn_bwd, BWD, _only(BWD, over)) == code


@pytest.mark.parametrize("over,code", HEADS + [
    (dict(S=None), 1), (dict(S_out=None), 1), (dict(o=None), 1), (dict(n=-1), 1), (dict(o=P(0x5000)), 1),
    (dict(S_out=P(0x1000)), 1), (dict(S=P(0x5004)), 1)])
def test_linear_attn_step_rejects(L, over, code):
    assert _call(L.mdn_linear_attn_step, STEP, _only(STEP, over)) == code


NORM = [(dict(x=None), 1), (dict(D=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(act=3), 1), (dict(dtype=7), 1),
        (dict(ld_x=15), 1), (dict(gate=P(0x8000), ld_g=15, dgate=P(0xb000)), 1), (dict(over=0, cu=P(0x9000), B=1), 1),
        (dict(D=16388, ld_x=16388, ld_dy=16388), 2), (dict(ws=None), 1), (dict(bytes=8), 1), (dict(w=P(0x8002)), 1)]


@pytest.mark.parametrize("over,code", NORM + BATCH + [
    (dict(y=None), 1), (dict(y=P(0x1000)), 1), (dict(stats=P(0xa004)), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1)])
def test_group_norm_fwd_rejects(L, over, code):
    assert _call(L.mdn_group_norm_fwd, GN, _only(GN, over)) == code


@pytest.mark.parametrize("over,code", NORM + BATCH + [
    (dict(stats=None), 1), (dict(stats=P(0x2004)), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dx=P(0x1000)), 1),
    (dict(gate=P(0x8000)), 1), (dict(ld_dy=15), 1), (dict(dw=P(0xa000), db=P(0xa000)), 1)])
def test_group_norm_bwd_rejects(L, over, code):
    assert _call(L.mdn_group_norm_bwd, GN_BWD, _only(GN_BWD, over)) == code


def test_sizes(L):
    f, b = L.mdn_linear_attn_fwd_workspace_size, L.mdn_linear_attn_bwd_workspace_size
    for g in (f, b):
        assert g(2, 5000, 4, 2, 16, 8, 1, 1) > 0 and g(2, 5000, 4, 2, 16, 8, 1, 1) % 256 == 0
        assert g(2, 5000, 3, 2, 16, 8, 1, 1) == 0 and g(2, 5000, 4, 2, 129, 8, 1, 1) == 0 and g(-1, 50, 4, 2, 16, 8, 1, 1) == 0
        assert g(2, 0, 4, 2, 16, 8, 1, 1) == 0
    # equal lengths that are not cut need none
    assert f(4, 400, 4, 2, 16, 8, 0, 1) == 0 and f(4, 400, 4, 2, 16, 8, 1, 1) > 0
    # shared heads' gradients by query head
    assert b(2, 5000, 4, 2, 16, 8, 1, 1) >= b(2, 5000, 4, 4, 16, 8, 1, 1) + 5000 * 4 * 24 * 4
    n = L.mdn_group_norm_fwd_workspace_size
    assert n(2, 100, 64, 4, 0, 1) == 0 and n(2, 100, 64, 4, 1, 1) > 0 and n(2, 100, 64, 5, 1, 1) == 0
    assert L.mdn_group_norm_bwd_workspace_size(2, 100, 64, 4, 0, 1) > 0
    assert L.mdn_group_norm_bwd_workspace_size(2, 100, 16385, 1, 0, 1) == 0


def test_binding_refuses():
    z = torch.zeros
    q, k, v, ld = z(1, 4, 4, 8), z(1, 4, 2, 8), z(1, 4, 2, 8), z(4)
    with pytest.raises(ValueError, match="CUDA"):
        mdn.linear_attn_fwd(q, k, v, ld)
    with pytest.raises(ValueError, match="CUDA"):
        mdn.linear_attn_step(q[0], k[0], v[0], ld, z(4, 4, 8, 8))
    with pytest.raises(TypeError):
        mdn.linear_attn_fwd(q.half(), k.half(), v.half(), ld)
    with pytest.raises(ValueError, match="CUDA"):
        mdn.group_norm_fwd(z(4, 8), 2)


def test_group_norm_arguments():
    from momentum_delta_rule_gb300 import attn
    x = torch.zeros(2, 3, 8)
    bad = [dict(groups=3), dict(groups=0), dict(groups=2.0), dict(groups=True), dict(activation="gelu"), dict(over="batch"),
           dict(cu_seqlens=torch.zeros(2, dtype=torch.int32))]
    for over in bad:
        kw = dict(dict(groups=2, activation="silu", over="token", cu_seqlens=None), **over)
        with pytest.raises(ValueError):
            attn._group_inputs(x, kw["groups"], None, None, None, kw["activation"], kw["over"], kw["cu_seqlens"], -1)
