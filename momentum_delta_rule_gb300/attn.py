"""Python binding of linear attention with a decay for each head and of the
group norm with an activation (``include/mdn.h``).

The conventions are those of the state-space layer's operators
(``momentum_delta_rule_gb300.ssm``): arguments are only marshalled, inputs may
be slices of a wider tensor with a constant stride between tokens, outputs and
workspaces are allocated on the stream the call runs on.
"""
import ctypes

import torch

import momentum_delta_rule_gb300 as _m

from .ssm import (_F32, _act, _address, _batch, _code, _dense, _elsewhere, _handle, _on, _raise, _required, _rows,
                  _size, _workspace)

_NORM_ACT = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}
_OVER = {"token": 0, "sequence": 1}


# --------------------------------------------------------- linear attention

# A small call takes 6 us on the GPU and 4 in the library: what is expected is
# looked at directly here, and only what does not fit goes through the checks
# that say what is wrong.

def _head_rows(name, t, B, T, H, d, dtype, index, step):
    """Elements between tokens of t, [B, T, H, d] (for a step [B, H, d], T = 1)."""
    s, width = t.stride(), H * d
    if t.dtype is dtype and t.get_device() == index and (s[-1] == 1 or d == 1) and (s[-2] == d or H == 1):
        if B * T <= 1:
            return width
        if T == 1:
            ld = s[0]
        else:
            ld = s[1]
            if B > 1 and s[0] != ld * T:
                ld = 0
        if ld >= width:
            return ld
    return _rows(name, t, (B, H, d) if step else (B, T, H, d), dtype, index, width, 2)


def _heads(q, k, v, log_decay, index, step):
    """Checks the tensors every form takes; (B, T, H, Hkv, dk, dv, code, addresses of
    q, k, v and log_decay, row strides)."""
    qs, n = q.shape, 3 if step else 4
    if len(qs) != n:
        raise ValueError("q must be [N, H, dk]" if step else "q must be [B, T, H, dk]")
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != n:
            raise ValueError("%s must be [..., heads, width] with the tokens of q" % name)
    ks, vs = k.shape, v.shape
    B, H, dk, Hkv, dv = qs[0], qs[-2], qs[-1], vs[-2], vs[-1]
    T = 1 if step else qs[1]
    if ks[0] != B or vs[0] != B or (not step and (ks[1] != T or vs[1] != T)):
        raise ValueError("k and v must have the tokens of q")
    if ks[-1] != dk or ks[-2] != Hkv:
        raise ValueError("k has heads %s, expected %s" % (tuple(ks[-2:]), (Hkv, dk)))
    if H == 0 or Hkv == 0 or dk == 0 or dv == 0 or H % Hkv:
        raise ValueError("the %d heads of q must be a multiple of the %d of v" % (H, Hkv))
    dtype = q.dtype
    code = _code(q)
    lds = (_head_rows("q", q, B, T, H, dk, dtype, index, step), _head_rows("k", k, B, T, Hkv, dk, dtype, index, step),
           _head_rows("v", v, B, T, Hkv, dv, dtype, index, step))
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _required("log_decay", log_decay, (H,), _F32, index))
    return B, T, H, Hkv, dk, dv, code, ptrs, lds


def _sequences(B, cu_seqlens, index):
    """(n_seq, address of cu_seqlens)"""
    if cu_seqlens is None:
        return B, None
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    return cu_seqlens.numel() - 1, _dense("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, index)


def linear_attn_fwd(q, k, v, log_decay, scale=1.0, S0=None, cu_seqlens=None, output_final_state=True, o=None, S_T=None,
                    workspace=None, stream=None):
    """Causal linear attention with a decay for each head over whole sequences
    (``mdn_linear_attn_fwd``): ``S_t = exp(log_decay) S_{t-1} + k_t v_t^T``,
    ``o_t = scale S_t^T q_t``.

    q ``[B, T, H, dk]``, k ``[B, T, Hkv, dk]``, v ``[B, T, Hkv, dv]`` in one
    dtype (packed: ``[1, sum T, ..]`` with ``cu_seqlens``), widths up to 128;
    consecutive query heads share a key and value head where Hkv < H.
    log_decay ``[H]`` fp32, at most zero; S0 ``[n_seq, H, dk, dv]`` fp32 or
    None.  Returns ``(o, S_T)`` (S_T None without ``output_final_state``).
    """
    if _elsewhere(q, "q", stream):
        with _on(q, stream):
            return linear_attn_fwd(q, k, v, log_decay, scale, S0, cu_seqlens, output_final_state, o, S_T, workspace)
    index = q.get_device()
    B, T, H, Hkv, dk, dv, code, ptrs, lds = _heads(q, k, v, log_decay, index, False)
    n_seq, cu = _sequences(B, cu_seqlens, index)
    state = (n_seq, H, dk, dv)
    s0 = _dense("S0", S0, state, _F32, index)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    else:
        _dense("o", o, (B, T, H, dv), q.dtype, index)
    if S_T is not None:
        _dense("S_T", S_T, state, _F32, index)
    elif output_final_state:
        S_T = torch.empty(state, dtype=_F32, device=q.device)
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_linear_attn_fwd_workspace_size", n_seq, B * T, H, Hkv, dk, dv, cu is not None, code), q.device,
        index)
    st = _m.lib().mdn_linear_attn_fwd(*ptrs, s0, o.data_ptr(), _address(S_T), cu, n_seq, B, T, H, Hkv, dk, dv, scale,
                                      *lds, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_linear_attn_fwd")
    return o, S_T


def linear_attn_bwd(q, k, v, log_decay, do, scale=1.0, S0=None, dS_T=None, cu_seqlens=None, need_dS0=None,
                    workspace=None, stream=None):
    """Gradient of ``linear_attn_fwd`` (``mdn_linear_attn_bwd``) from its inputs,
    the adjoint do of o and optionally ``dS_T`` of the final states.  Returns a
    dict with dq, dk, dv and dS0 (None unless ``need_dS0``, by default where
    S0 was given).  The decays are constants and have no gradient."""
    if _elsewhere(q, "q", stream):
        with _on(q, stream):
            return linear_attn_bwd(q, k, v, log_decay, do, scale, S0, dS_T, cu_seqlens, need_dS0, workspace)
    index = q.get_device()
    B, T, H, Hkv, dk, dv, code, ptrs, lds = _heads(q, k, v, log_decay, index, False)
    n_seq, cu = _sequences(B, cu_seqlens, index)
    if not isinstance(do, torch.Tensor) or do.shape != (B, T, H, dv):
        _required("do", do, (B, T, H, dv), q.dtype, index)
    ld_do = _head_rows("do", do, B, T, H, dv, q.dtype, index, False)
    state = (n_seq, H, dk, dv)
    s0 = _dense("S0", S0, state, _F32, index)
    dsT = _dense("dS_T", dS_T, state, _F32, index)
    if need_dS0 is None:
        need_dS0 = S0 is not None
    dev, dtype = q.device, q.dtype
    g = {"dq": torch.empty((B, T, H, dk), dtype=dtype, device=dev), "dk": torch.empty((B, T, Hkv, dk), dtype=dtype, device=dev),
         "dv": torch.empty((B, T, Hkv, dv), dtype=dtype, device=dev),
         "dS0": torch.empty(state, dtype=_F32, device=dev) if need_dS0 else None}
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_linear_attn_bwd_workspace_size", n_seq, B * T, H, Hkv, dk, dv, cu is not None, code), q.device,
        index)
    st = _m.lib().mdn_linear_attn_bwd(*ptrs, s0, do.data_ptr(), dsT, *map(_address, g.values()), cu, n_seq, B, T, H, Hkv,
                                      dk, dv, scale, *lds, ld_do, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_linear_attn_bwd")
    return g


def linear_attn_step(q, k, v, log_decay, S, scale=1.0, S_out=None, o=None, stream=None):
    """One token per sequence (``mdn_linear_attn_step``): q ``[N, H, dk]``, k
    ``[N, Hkv, dk]``, v ``[N, Hkv, dv]``; S ``[N, H, dk, dv]`` fp32 is updated in
    place or into ``S_out``.  Returns o ``[N, H, dv]``."""
    if _elsewhere(q, "q", stream):
        with _on(q, stream):
            return linear_attn_step(q, k, v, log_decay, S, scale, S_out, o)
    index = q.get_device()
    n, _, H, Hkv, dk, dv, code, ptrs, lds = _heads(q, k, v, log_decay, index, True)
    s0 = _required("S", S, (n, H, dk, dv), _F32, index)
    so = s0 if S_out is None else _dense("S_out", S_out, (n, H, dk, dv), _F32, index)
    if o is None:
        o = torch.empty((n, H, dv), dtype=q.dtype, device=q.device)
    else:
        _dense("o", o, (n, H, dv), q.dtype, index)
    st = _m.lib().mdn_linear_attn_step(*ptrs, s0, so, o.data_ptr(), n, H, Hkv, dk, dv, scale, *lds, code, _handle(index))
    if st:
        _raise(st, "mdn_linear_attn_step")
    return o


# --------------------------------------------------------------- group norm

def _group_rows(name, t, like, D, dtype, index):
    """Elements between tokens of t, which has the shape of `like`, [..., D]."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == like.shape:
        if t.is_contiguous():
            return D
        s, n = t.stride(), t.dim()
        if s[-1] == 1 and n == 2 and s[0] >= D:
            return s[0]
        if s[-1] == 1 and n == 3 and s[1] >= D and t.shape[1] > 1 and (t.shape[0] == 1 or s[0] == s[1] * t.shape[1]):
            return s[1]
    return _rows(name, t, like.shape, dtype, index, D)


def _group_inputs(x, groups, weight, bias, gate, activation, over, cu_seqlens, index):
    """Checks what both directions take; (batch, D, code, addresses, row strides,
    over, act)."""
    over = _act(_OVER, "over", over)
    act = _act(_NORM_ACT, "activation", activation)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x must be [..., D] with at least one channel")
    D = x.shape[-1]
    if isinstance(groups, bool) or not isinstance(groups, int) or groups < 1 or D % groups:
        raise ValueError("groups must divide the %d channels of x" % D)
    if over:
        B, T, _, n_seq, cu = _batch(x, cu_seqlens, index, "x")
    else:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens is for norms over a sequence")
        B, T, n_seq, cu = 1, x.numel() // D, 1, None
        if T > 0x3fffffff:
            raise ValueError("x has more than 2^30 - 1 rows")
    dtype, code = x.dtype, _code(x)
    lds = (_group_rows("x", x, x, D, dtype, index), _group_rows("gate", gate, x, D, dtype, index) if gate is not None else 0)
    ptrs = (x.data_ptr(), _address(gate), _dense("weight", weight, (D,), _F32, index),
            _dense("bias", bias, (D,), _F32, index))
    return (cu, n_seq, B, T), D, code, ptrs, lds, over, act


def _stats_shape(x, groups, over, n_seq):
    return (n_seq, groups, 2) if over else x.shape[:-1] + (groups, 2)


def group_norm_fwd(x, groups, weight=None, bias=None, gate=None, activation=None, over="token", center=True,
                   cu_seqlens=None, eps=1e-5, return_stats=False, y=None, workspace=None, stream=None):
    """Group norm with an activation, channels last (``mdn_group_norm_fwd``):
    ``u = (x - mean) / sqrt(var + eps) * weight + bias`` and ``y = act(u)``, or
    with a gate ``y = u * act(gate)``.

    x and gate ``[..., D]`` in one dtype; weight and bias ``[D]`` fp32 or None;
    activation "silu", "sigmoid" or None.  A group is ``D / groups``
    neighbouring channels of one token (``over="token"``, the norm of each
    head's output), or of a whole sequence (``over="sequence"``: x ``[B, T, D]``,
    or packed ``[1, sum T, D]`` with ``cu_seqlens``).  Without ``center`` the
    mean is not taken away (a root-mean-square norm).  Returns y, and with
    ``return_stats`` second the fp32 mean and factor of every group (``[..., groups,
    2]`` or ``[n_seq, groups, 2]``), which ``group_norm_bwd`` takes.
    """
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return group_norm_fwd(x, groups, weight, bias, gate, activation, over, center, cu_seqlens, eps, return_stats,
                                  y, workspace)
    index = x.get_device()
    batch, D, code, ptrs, lds, over, act = _group_inputs(x, groups, weight, bias, gate, activation, over, cu_seqlens, index)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _dense("y", y, x.shape, x.dtype, index)
    stats = None
    if return_stats:
        stats = torch.empty(_stats_shape(x, groups, over, batch[1]), dtype=_F32, device=x.device)
    need = _size("mdn_group_norm_fwd_workspace_size", batch[1], batch[2] * batch[3], D, groups, over, code) if over else 0
    workspace, ws, nbytes = _workspace(workspace, need, x.device, index)
    st = _m.lib().mdn_group_norm_fwd(*ptrs, y.data_ptr(), _address(stats), *batch, D, groups, over, 1 if center else 0,
                                     act, eps, *lds, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_group_norm_fwd")
    return (y, stats) if return_stats else y


def group_norm_bwd(x, groups, stats, dy, weight=None, bias=None, gate=None, activation=None, over="token", center=True,
                   cu_seqlens=None, eps=1e-5, workspace=None, stream=None):
    """Gradient of ``group_norm_fwd`` (``mdn_group_norm_bwd``) from its inputs, its
    stats and the adjoint dy of y.  ``eps`` is accepted for symmetry; the stats
    already hold it.  Returns a dict with dx, dgate, dw and dbias (None where
    the input is None)."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return group_norm_bwd(x, groups, stats, dy, weight, bias, gate, activation, over, center, cu_seqlens, eps,
                                  workspace)
    index = x.get_device()
    batch, D, code, ptrs, lds, over, act = _group_inputs(x, groups, weight, bias, gate, activation, over, cu_seqlens, index)
    st2 = _required("stats", stats, _stats_shape(x, groups, over, batch[1]), _F32, index)
    ld_dy = _group_rows("dy", dy, x, D, x.dtype, index)
    dev, dtype, shape = x.device, x.dtype, x.shape
    g = {"dx": torch.empty(shape, dtype=dtype, device=dev),
         "dgate": torch.empty(shape, dtype=dtype, device=dev) if gate is not None else None,
         "dw": torch.empty_like(weight) if weight is not None else None,
         "dbias": torch.empty_like(bias) if bias is not None else None}
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_group_norm_bwd_workspace_size", batch[1], batch[2] * batch[3], D, groups, over, code), x.device,
        index)
    st = _m.lib().mdn_group_norm_bwd(*ptrs, st2, dy.data_ptr(), *map(_address, g.values()), *batch, D, groups, over,
                                     1 if center else 0, act, *lds, ld_dy, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_group_norm_bwd")
    return g


def declare(L):
    """Argument and result types of this part of the C ABI."""
    vp, ci, cl, cs, cf = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float)
    for name, res, args in (
            ("mdn_linear_attn_fwd_workspace_size", cs, [ci] * 8),
            ("mdn_linear_attn_bwd_workspace_size", cs, [ci] * 8),
            ("mdn_linear_attn_fwd", ci, [vp] * 8 + [ci] * 7 + [cf] + [cl] * 3 + [ci, vp, cs, vp]),
            ("mdn_linear_attn_bwd", ci, [vp] * 12 + [ci] * 7 + [cf] + [cl] * 4 + [ci, vp, cs, vp]),
            ("mdn_linear_attn_step", ci, [vp] * 7 + [ci] * 5 + [cf] + [cl] * 3 + [ci, vp]),
            ("mdn_group_norm_fwd_workspace_size", cs, [ci] * 6),
            ("mdn_group_norm_bwd_workspace_size", cs, [ci] * 6),
            ("mdn_group_norm_fwd", ci, [vp] * 7 + [ci] * 8 + [cf] + [cl] * 2 + [ci, vp, cs, vp]),
            ("mdn_group_norm_bwd", ci, [vp] * 11 + [ci] * 8 + [cl] * 3 + [ci, vp, cs, vp])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
