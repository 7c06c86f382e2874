"""Python binding of the state-space layer's operators (``include/mdn.h``):
the short causal convolution, the selective scan and the norms around a block.

Like the rest of the binding it only marshals arguments.  Inputs that are
rows of channels may be slices of a wider tensor (for example the halves of an
input projection): their last dimension is contiguous and their tokens lie a
constant stride apart.  Outputs and workspaces are allocated on the stream the
call runs on.
"""
import contextlib
import ctypes

import torch

import momentum_delta_rule_gb300 as _m

MDN_SSM_CHUNK = 32
_CONV_ACT = {None: 0, "none": 0, "silu": 1}
_GATE_ACT = {"sigmoid": 0, "silu": 1}


def _on(dev, stream):
    """Makes `stream` (or the current one) of `dev` the current stream."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() == dev.index:
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _handle(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _row_stride(name, t, tail):
    """Elements between rows of t, whose last `tail` dimensions are a row."""
    shape, stride = t.shape, t.stride()
    width = 1
    for d in range(t.dim() - 1, t.dim() - 1 - tail, -1):
        if shape[d] != 1 and stride[d] != width:
            raise ValueError("%s: the last %d dimension(s) must be contiguous" % (name, tail))
        width *= shape[d]
    if t.numel() == 0:
        return width
    ld = span = None
    for d in range(t.dim() - 1 - tail, -1, -1):
        if shape[d] == 1:
            continue
        if ld is None:
            ld, span = stride[d], stride[d] * shape[d]
        elif stride[d] != span:
            raise ValueError("%s: its rows must lie a constant stride apart" % name)
        else:
            span *= shape[d]
    if ld is None:
        return width
    if ld < width:
        raise ValueError("%s: its rows overlap" % name)
    return ld


def _rows(name, t, shape, dtype, dev, tail=1):
    """Checks a rows input and returns its row stride."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return _row_stride(name, t, tail)


def _dense(name, t, shape, dtype, dev):
    """Checks a dense tensor (None passes)."""
    if t is None:
        return
    _m._check_cuda(name, t, dtype, dev)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _empty(given, name, shape, dtype, dev):
    if given is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _dense(name, given, torch.Size(shape), dtype, dev)
    return given


def _workspace(given, need, dev):
    if given is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _m._check_cuda("workspace", given, torch.uint8, dev)
    return given


def _batch(x, cu_seqlens, dev, what):
    if x.dim() != 3:
        raise ValueError("%s must be [B, T, D]" % what)
    B, T, D = x.shape
    if cu_seqlens is None:
        return B, T, D, B
    _m._check_cuda("cu_seqlens", cu_seqlens, torch.int32, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    return B, T, D, cu_seqlens.numel() - 1


def _act(table, name, value):
    if value not in table:
        raise ValueError("%s must be one of %s" % (name, sorted(map(str, table))))
    return table[value]


def _raise_unless_ok(st, where):
    if st != _m.MDN_OK:
        raise _m.MdnError(st, where)


# ------------------------------------------------------------ convolution

def short_conv_fwd(x, weight, bias=None, state=None, cu_seqlens=None, activation="silu",
                   output_final_state=False, y=None, state_T=None, stream=None):
    """Causal depthwise convolution along the tokens (``mdn_short_conv_fwd``).

    x ``[B, T, D]`` (or packed ``[1, sum T, D]`` with ``cu_seqlens``); weight
    ``[D, width]`` and bias ``[D]`` fp32, width 2 to 4 (the last tap meets the
    current token); state ``[n_seq, width - 1, D]`` in the dtype of x, the
    tokens before each sequence (None: zeros); activation "silu" or None.
    Returns ``(y, state_T)``; ``state_T`` is None unless asked for.
    """
    L = _m.lib()
    dev = x.device
    B, T, D, n_seq = _batch(x, cu_seqlens, dev, "x")
    code = _m._dtype_code(x.dtype)
    ld_x = _rows("x", x, x.shape, x.dtype, dev)
    W = _conv_params(weight, bias, D, dev)
    _dense("state", state, (n_seq, W - 1, D), x.dtype, dev)
    act = _act(_CONV_ACT, "activation", activation)
    with _on(dev, stream):
        y = _empty(y, "y", (B, T, D), x.dtype, dev)
        if output_final_state or state_T is not None:
            state_T = _empty(state_T, "state_T", (n_seq, W - 1, D), x.dtype, dev)
        st = L.mdn_short_conv_fwd(
            x.data_ptr(), weight.data_ptr(), _m._ptr(bias), _m._ptr(state), y.data_ptr(),
            _m._ptr(state_T), _m._ptr(cu_seqlens), n_seq, B, T, D, W, act, ld_x, code, _handle(dev))
    _raise_unless_ok(st, "mdn_short_conv_fwd")
    return y, state_T


def _conv_params(weight, bias, D, dev):
    _m._check_cuda("weight", weight, torch.float32, dev)
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError("weight must be [D, width]")
    _dense("bias", bias, (D,), torch.float32, dev)
    return weight.shape[1]


def short_conv_bwd(x, weight, dy, bias=None, state=None, cu_seqlens=None, activation="silu",
                   dstate_T=None, need_dstate=None, workspace=None, stream=None):
    """Gradient of ``short_conv_fwd`` (``mdn_short_conv_bwd``) from its inputs,
    the adjoint dy of y and optionally ``dstate_T`` of the final state.
    Returns a dict with dx, dw, dbias (None without a bias) and dstate (None
    unless ``need_dstate``, by default where a state was given)."""
    L = _m.lib()
    dev = x.device
    B, T, D, n_seq = _batch(x, cu_seqlens, dev, "x")
    code = _m._dtype_code(x.dtype)
    ld_x = _rows("x", x, x.shape, x.dtype, dev)
    ld_dy = _rows("dy", dy, x.shape, x.dtype, dev)
    W = _conv_params(weight, bias, D, dev)
    _dense("state", state, (n_seq, W - 1, D), x.dtype, dev)
    _dense("dstate_T", dstate_T, (n_seq, W - 1, D), x.dtype, dev)
    act = _act(_CONV_ACT, "activation", activation)
    need = int(L.mdn_short_conv_bwd_workspace_size(B * T, D, W, code))
    if need_dstate is None:
        need_dstate = state is not None
    with _on(dev, stream):
        g = {"dx": torch.empty((B, T, D), dtype=x.dtype, device=dev),
             "dw": torch.empty_like(weight),
             "dbias": torch.empty_like(bias) if bias is not None else None,
             "dstate": (torch.empty((n_seq, W - 1, D), dtype=x.dtype, device=dev)
                        if need_dstate else None)}
        workspace = _workspace(workspace, need, dev)
        st = L.mdn_short_conv_bwd(
            x.data_ptr(), weight.data_ptr(), _m._ptr(bias), _m._ptr(state), dy.data_ptr(),
            _m._ptr(dstate_T), g["dx"].data_ptr(), g["dw"].data_ptr(), _m._ptr(g["dbias"]),
            _m._ptr(g["dstate"]), _m._ptr(cu_seqlens), n_seq, B, T, D, W, act, ld_x, ld_dy, code,
            workspace.data_ptr(), workspace.numel(), _handle(dev))
    _raise_unless_ok(st, "mdn_short_conv_bwd")
    return g


def short_conv_step(x, weight, state, bias=None, activation="silu", state_out=None, y=None,
                    stream=None):
    """One new token per sequence (``mdn_short_conv_step``): x ``[N, D]``, state
    ``[N, width - 1, D]``, shifted by the token in place or into ``state_out``.
    Returns y ``[N, D]``."""
    L = _m.lib()
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    N, D = x.shape
    dev = x.device
    code = _m._dtype_code(x.dtype)
    ld_x = _rows("x", x, x.shape, x.dtype, dev)
    W = _conv_params(weight, bias, D, dev)
    _dense("state", state, (N, W - 1, D), x.dtype, dev)
    if state_out is None:
        state_out = state
    else:
        _dense("state_out", state_out, (N, W - 1, D), x.dtype, dev)
    act = _act(_CONV_ACT, "activation", activation)
    with _on(dev, stream):
        y = _empty(y, "y", (N, D), x.dtype, dev)
        st = L.mdn_short_conv_step(x.data_ptr(), weight.data_ptr(), _m._ptr(bias), state.data_ptr(),
                                   state_out.data_ptr(), y.data_ptr(), N, D, W, act, ld_x, code,
                                   _handle(dev))
    _raise_unless_ok(st, "mdn_short_conv_step")
    return y


# ------------------------------------------------------------------- scan

def ssm_state_slots(n_seq, B, T, packed):
    """Slots of the saved states (``mdn_ssm_state_slots``): chunk c of 32 tokens
    of sequence s at slot s * ceil(T / 32) + c, or, packed, at
    sum_{s' < s} ceil(L_s' / 32) + c."""
    return int(_m.lib().mdn_ssm_state_slots(int(n_seq), int(B), int(T), 1 if packed else 0))


def _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, lead, D, dev):
    """Checks the tensors every form of the scan takes; (G, N, row strides)."""
    shape = u.shape
    if Bm.dim() != len(lead) + 2:
        raise ValueError("Bm must be [%s, G, N]" % ", ".join(["N"] if len(lead) == 1 else ["B", "T"]))
    G, N = Bm.shape[-2:]
    bc = torch.Size(tuple(lead) + (G, N))
    lds = (_rows("u", u, shape, u.dtype, dev), _rows("dt", dt, shape, u.dtype, dev),
           _rows("Bm", Bm, bc, u.dtype, dev, tail=2), _rows("Cm", Cm, bc, u.dtype, dev, tail=2),
           _rows("z", z, shape, u.dtype, dev) if z is not None else 0)
    _dense("A", A, (D, N), torch.float32, dev)
    _dense("D_skip", D_skip, (D,), torch.float32, dev)
    _dense("dt_bias", dt_bias, (D,), torch.float32, dev)
    return G, N, lds


def ssm_scan_fwd(u, dt, A, Bm, Cm, D_skip=None, z=None, dt_bias=None, softplus=True, h0=None,
                 cu_seqlens=None, output_final_state=True, return_chunk_states=False, y=None,
                 h_T=None, workspace=None, stream=None):
    """Selective scan over whole sequences (``mdn_ssm_scan_fwd``).

    u, dt, z ``[B, T, D]`` and Bm, Cm ``[B, T, G, N]`` in one dtype (packed:
    ``[1, sum T, ..]`` with ``cu_seqlens``); A ``[D, N]``, D_skip ``[D]``,
    dt_bias ``[D]`` fp32; h0 ``[n_seq, D, N]`` fp32 or None.  N up to 128, G
    divides D.  Returns ``(y, h_T)`` (h_T None without ``output_final_state``),
    and with ``return_chunk_states`` third the states before every 32nd token,
    ``[ssm_state_slots(...), D, N]`` fp32, which ``ssm_scan_bwd`` takes.
    """
    L = _m.lib()
    dev = u.device
    B, T, D, n_seq = _batch(u, cu_seqlens, dev, "u")
    code = _m._dtype_code(u.dtype)
    G, N, lds = _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, (B, T), D, dev)
    _dense("h0", h0, (n_seq, D, N), torch.float32, dev)
    need = int(L.mdn_ssm_scan_fwd_workspace_size(n_seq, B * T, D, G, N, code))
    h_chunks = None
    with _on(dev, stream):
        y = _empty(y, "y", (B, T, D), u.dtype, dev)
        if output_final_state or h_T is not None:
            h_T = _empty(h_T, "h_T", (n_seq, D, N), torch.float32, dev)
        if return_chunk_states:
            slots = ssm_state_slots(n_seq, B, T, cu_seqlens is not None)
            h_chunks = torch.empty((slots, D, N), dtype=torch.float32, device=dev)
        workspace = _workspace(workspace, need, dev)
        st = L.mdn_ssm_scan_fwd(
            u.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
            _m._ptr(D_skip), _m._ptr(z), _m._ptr(dt_bias), _m._ptr(h0), y.data_ptr(), _m._ptr(h_T),
            _m._ptr(h_chunks), _m._ptr(cu_seqlens), n_seq, B, T, D, G, N, 1 if softplus else 0,
            *lds, code, workspace.data_ptr(), workspace.numel(), _handle(dev))
    _raise_unless_ok(st, "mdn_ssm_scan_fwd")
    return (y, h_T, h_chunks) if return_chunk_states else (y, h_T)


def ssm_scan_bwd(u, dt, A, Bm, Cm, h_chunks, dy, D_skip=None, z=None, dt_bias=None, softplus=True,
                 cu_seqlens=None, dh_T=None, need_dh0=False, workspace=None, stream=None):
    """Gradient of ``ssm_scan_fwd`` (``mdn_ssm_scan_bwd``) from its inputs, its
    chunk states (``return_chunk_states=True``), the adjoint dy of y and
    optionally ``dh_T`` of the final states.  Returns a dict with du, ddt, dA,
    dB, dC, dD_skip, dz, ddt_bias and dh0 (None where the input is None, dh0
    unless ``need_dh0``)."""
    L = _m.lib()
    dev = u.device
    B, T, D, n_seq = _batch(u, cu_seqlens, dev, "u")
    code = _m._dtype_code(u.dtype)
    G, N, lds = _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, (B, T), D, dev)
    ld_dy = _rows("dy", dy, u.shape, u.dtype, dev)
    slots = ssm_state_slots(n_seq, B, T, cu_seqlens is not None)
    _dense("h_chunks", h_chunks, (slots, D, N), torch.float32, dev)
    _dense("dh_T", dh_T, (n_seq, D, N), torch.float32, dev)
    need = int(L.mdn_ssm_scan_bwd_workspace_size(n_seq, B * T, D, G, N, code))
    with _on(dev, stream):
        g = {"du": torch.empty((B, T, D), dtype=u.dtype, device=dev),
             "ddt": torch.empty((B, T, D), dtype=u.dtype, device=dev),
             "dA": torch.empty((D, N), dtype=torch.float32, device=dev),
             "dB": torch.empty((B, T, G, N), dtype=u.dtype, device=dev),
             "dC": torch.empty((B, T, G, N), dtype=u.dtype, device=dev),
             "dD_skip": torch.empty_like(D_skip) if D_skip is not None else None,
             "dz": torch.empty((B, T, D), dtype=u.dtype, device=dev) if z is not None else None,
             "ddt_bias": torch.empty_like(dt_bias) if dt_bias is not None else None,
             "dh0": (torch.empty((n_seq, D, N), dtype=torch.float32, device=dev)
                     if need_dh0 else None)}
        workspace = _workspace(workspace, need, dev)
        st = L.mdn_ssm_scan_bwd(
            u.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
            _m._ptr(D_skip), _m._ptr(z), _m._ptr(dt_bias), h_chunks.data_ptr(), dy.data_ptr(),
            _m._ptr(dh_T), g["du"].data_ptr(), g["ddt"].data_ptr(), g["dA"].data_ptr(),
            g["dB"].data_ptr(), g["dC"].data_ptr(), _m._ptr(g["dD_skip"]), _m._ptr(g["dz"]),
            _m._ptr(g["ddt_bias"]), _m._ptr(g["dh0"]), _m._ptr(cu_seqlens), n_seq, B, T, D, G, N,
            1 if softplus else 0, *lds, ld_dy, code, workspace.data_ptr(), workspace.numel(),
            _handle(dev))
    _raise_unless_ok(st, "mdn_ssm_scan_bwd")
    return g


def ssm_scan_step(u, dt, A, Bm, Cm, h, D_skip=None, z=None, dt_bias=None, softplus=True,
                  h_out=None, y=None, stream=None):
    """One token per sequence (``mdn_ssm_scan_step``): u, dt, z ``[N, D]``, Bm, Cm
    ``[N, G, n_states]``; h ``[N, D, n_states]`` fp32 is updated in place or
    into ``h_out``.  Returns y ``[N, D]``."""
    L = _m.lib()
    if u.dim() != 2:
        raise ValueError("u must be [N, D]")
    n, D = u.shape
    dev = u.device
    code = _m._dtype_code(u.dtype)
    G, N, lds = _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, (n,), D, dev)
    _dense("h", h, (n, D, N), torch.float32, dev)
    if h_out is None:
        h_out = h
    else:
        _dense("h_out", h_out, (n, D, N), torch.float32, dev)
    with _on(dev, stream):
        y = _empty(y, "y", (n, D), u.dtype, dev)
        st = L.mdn_ssm_scan_step(
            u.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
            _m._ptr(D_skip), _m._ptr(z), _m._ptr(dt_bias), h.data_ptr(), h_out.data_ptr(),
            y.data_ptr(), n, D, G, N, 1 if softplus else 0, *lds, code, _handle(dev))
    _raise_unless_ok(st, "mdn_ssm_scan_step")
    return y


# ------------------------------------------------------------------ norms

def _norm_inputs(y, x, gate, w_post, w_pre, scale, gate_act):
    if y.dim() < 1:
        raise ValueError("y must be [..., D]")
    dev, D = y.device, y.shape[-1]
    lds = (_rows("y", y, y.shape, y.dtype, dev), _rows("x", x, y.shape, y.dtype, dev),
           _rows("gate", gate, y.shape, y.dtype, dev) if gate is not None else 0)
    for name, t in (("w_post", w_post), ("w_pre", w_pre), ("scale", scale)):
        _dense(name, t, (D,), torch.float32, dev)
    if D == 0:
        raise ValueError("y must have at least one column")
    return dev, D, y.numel() // D, lds, _act(_GATE_ACT, "gate_act", gate_act)


def norm_residual_fwd(y, x, w_post=None, w_pre=None, gate=None, gate_act="sigmoid", scale=None,
                      eps=1e-6, return_stats=False, x_out=None, stream=None):
    """The end of a block and the start of the next (``mdn_norm_residual_fwd``):
    ``x_out = x + scale * RMSNorm(y) * w_post * act(gate)`` and
    ``h = RMSNorm(x_out) * w_pre``, rows of the last dimension.

    y (the block's output), x (the residual) and gate share a dtype; w_post,
    w_pre, scale ``[D]`` fp32, each optional (no norm of y, no h, no scale).
    ``x_out`` may be x.  Returns ``(x_out, h)``, and with ``return_stats``
    third the ``[..., 2]`` fp32 factors the gradient takes.
    """
    L = _m.lib()
    dev, D, rows, lds, act = _norm_inputs(y, x, gate, w_post, w_pre, scale, gate_act)
    code = _m._dtype_code(y.dtype)
    h = stats = None
    with _on(dev, stream):
        x_out = _empty(x_out, "x_out", y.shape, y.dtype, dev)
        if w_pre is not None:
            h = torch.empty(y.shape, dtype=y.dtype, device=dev)
        if return_stats:
            stats = torch.empty(y.shape[:-1] + (2,), dtype=torch.float32, device=dev)
        st = L.mdn_norm_residual_fwd(
            y.data_ptr(), x.data_ptr(), _m._ptr(gate), _m._ptr(w_post), _m._ptr(w_pre),
            _m._ptr(scale), x_out.data_ptr(), _m._ptr(h), _m._ptr(stats), rows, D, act, eps, *lds,
            code, _handle(dev))
    _raise_unless_ok(st, "mdn_norm_residual_fwd")
    return (x_out, h, stats) if return_stats else (x_out, h)


def norm_residual_bwd(y, x, stats, dx_out, dh=None, w_post=None, w_pre=None, gate=None,
                      gate_act="sigmoid", scale=None, eps=1e-6, workspace=None, stream=None):
    """Gradient of ``norm_residual_fwd`` (``mdn_norm_residual_bwd``) from its
    inputs, its stats and the adjoints of x_out and h.  ``eps`` is accepted for
    symmetry; the stats already hold it.  Returns a dict with dy, dx, dgate,
    dw_post, dw_pre and dscale (None where the input is None)."""
    L = _m.lib()
    dev, D, rows, lds, act = _norm_inputs(y, x, gate, w_post, w_pre, scale, gate_act)
    code = _m._dtype_code(y.dtype)
    _dense("stats", stats, y.shape[:-1] + (2,), torch.float32, dev)
    ld_dx_out = _rows("dx_out", dx_out, y.shape, y.dtype, dev)
    if w_pre is not None and dh is None:
        raise ValueError("dh is required with w_pre")
    ld_dh = _rows("dh", dh, y.shape, y.dtype, dev) if dh is not None else 0
    need = int(L.mdn_norm_residual_bwd_workspace_size(rows, D, code))
    with _on(dev, stream):
        new = lambda like: torch.empty_like(like) if like is not None else None
        rows_new = lambda: torch.empty(y.shape, dtype=y.dtype, device=dev)
        g = {"dy": rows_new(), "dx": rows_new(), "dgate": rows_new() if gate is not None else None,
             "dw_post": new(w_post), "dw_pre": new(w_pre), "dscale": new(scale)}
        workspace = _workspace(workspace, need, dev)
        st = L.mdn_norm_residual_bwd(
            y.data_ptr(), x.data_ptr(), _m._ptr(gate), _m._ptr(w_post), _m._ptr(w_pre),
            _m._ptr(scale), stats.data_ptr(), dx_out.data_ptr(), _m._ptr(dh), g["dy"].data_ptr(),
            g["dx"].data_ptr(), _m._ptr(g["dgate"]), _m._ptr(g["dw_post"]), _m._ptr(g["dw_pre"]),
            _m._ptr(g["dscale"]), rows, D, act, *lds, ld_dx_out, ld_dh, code, workspace.data_ptr(),
            workspace.numel(), _handle(dev))
    _raise_unless_ok(st, "mdn_norm_residual_bwd")
    return g


def declare(L):
    """Argument and result types of this part of the C ABI."""
    vp, ci, cl, cs, cf = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                          ctypes.c_float)
    for name, res, args in (
            ("mdn_short_conv_fwd", ci, [vp] * 7 + [ci] * 6 + [cl, ci, vp]),
            ("mdn_short_conv_bwd_workspace_size", cs, [ci] * 4),
            ("mdn_short_conv_bwd", ci, [vp] * 11 + [ci] * 6 + [cl] * 2 + [ci, vp, cs, vp]),
            ("mdn_short_conv_step", ci, [vp] * 6 + [ci] * 4 + [cl, ci, vp]),
            ("mdn_ssm_state_slots", cs, [ci] * 4),
            ("mdn_ssm_scan_fwd_workspace_size", cs, [ci] * 6),
            ("mdn_ssm_scan_bwd_workspace_size", cs, [ci] * 6),
            ("mdn_ssm_scan_fwd", ci, [vp] * 13 + [ci] * 7 + [cl] * 5 + [ci, vp, cs, vp]),
            ("mdn_ssm_scan_bwd", ci, [vp] * 21 + [ci] * 7 + [cl] * 6 + [ci, vp, cs, vp]),
            ("mdn_ssm_scan_step", ci, [vp] * 11 + [ci] * 5 + [cl] * 5 + [ci, vp]),
            ("mdn_norm_residual_fwd", ci, [vp] * 9 + [ci] * 3 + [cf] + [cl] * 3 + [ci, vp]),
            ("mdn_norm_residual_bwd_workspace_size", cs, [ci] * 3),
            ("mdn_norm_residual_bwd", ci, [vp] * 15 + [ci] * 3 + [cl] * 5 + [ci, vp, cs, vp])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
