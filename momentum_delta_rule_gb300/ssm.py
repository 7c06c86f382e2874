"""Python binding of the state-space layer's operators (``include/mdn.h``):
the short causal convolution, the selective scan and the norms around a block.

Like the rest of the binding it only marshals arguments.  Inputs that are
rows of channels may be slices of a wider tensor (for example the halves of an
input projection): their last dimension is contiguous and their tokens lie a
constant stride apart.  Outputs and workspaces are allocated on the stream the
call runs on.
"""
import ctypes
import functools

import torch

import momentum_delta_rule_gb300 as _m

MDN_SSM_CHUNK = 32
_CONV_ACT = {None: 0, "none": 0, "silu": 1}
_GATE_ACT = {"sigmoid": 0, "silu": 1}
_CODES = {torch.float32: _m.MDN_F32, torch.bfloat16: _m.MDN_BF16}
_F32, _U8 = torch.float32, torch.uint8

# Small calls take a few microseconds on the GPU, so the checks below first
# test for what is expected, without building anything, and only then find out
# what is wrong.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(index):
    """The current stream of a device, as the C ABI takes it."""
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _elsewhere(t, name, stream):
    """Whether a call on t has to change the current device or stream first."""
    index = t.get_device()
    if index < 0:
        _code(t)
        raise ValueError("%s must be a CUDA tensor" % name)
    return stream is not None or torch.cuda.current_device() != index


def _on(t, stream):
    """Makes the call's device, and its stream where one is given, the current one."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream)


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


def _refuse(name, t, shape, dtype, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor, got %s" % (name, type(t).__name__))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    raise ValueError("%s must be contiguous" % name)


def _rows(name, t, shape, dtype, index, width, tail=1):
    """Checks a rows input and returns its row stride (`width`: of a dense row)."""
    if t is None or t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _refuse(name, t, shape, dtype, index)
    if t.is_contiguous():
        return width
    # a slice of [.., T, wider] rows
    st = t.stride()
    lead = len(st) - tail
    if (lead <= 2 and st[-1] == 1 and (tail == 1 or shape[-2] == 1 or st[-2] == shape[-1])
            and (lead == 1 or shape[0] == 1 or st[0] == st[1] * shape[1])):
        ld = st[lead - 1]
        if ld >= width and shape[lead - 1] > 1:
            return ld
    return _row_stride(name, t, tail)


def _dense(name, t, shape, dtype, index):
    """Checks a dense tensor and returns its address (None passes)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, shape, dtype, index)
    return t.data_ptr()


def _required(name, t, shape, dtype, index):
    if t is None:
        _refuse(name, t, shape, dtype, index)
    return _dense(name, t, shape, dtype, index)


def _new(given, name, shape, dtype, dev, index):
    if given is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _dense(name, given, shape, dtype, index)
    return given


def _address(t):
    return None if t is None else t.data_ptr()


def _code(t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("tensors must be float32 or bfloat16, got %s" % t.dtype)
    return code


@functools.lru_cache(maxsize=4096)
def _size(which, *sizes):
    """A size the library computes from sizes alone."""
    return int(getattr(_m.lib(), which)(*sizes))


def _workspace(given, need, dev, index):
    """(tensor, address, bytes) of a call's workspace."""
    if given is None:
        if need == 0:
            return None, None, 0
        given = torch.empty(need, dtype=_U8, device=dev)
    elif given.dtype is not _U8 or given.get_device() != index or not given.is_contiguous():
        _refuse("workspace", given, given.shape, _U8, index)
    return given, given.data_ptr(), given.numel()


def _batch(x, cu_seqlens, index, what):
    if x.dim() != 3:
        raise ValueError("%s must be [B, T, D]" % what)
    B, T, D = x.shape
    if cu_seqlens is None:
        return B, T, D, B, None
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    return B, T, D, cu_seqlens.numel() - 1, _dense("cu_seqlens", cu_seqlens, cu_seqlens.shape,
                                                   torch.int32, index)


def _act(table, name, value):
    act = table.get(value)
    if act is None:
        raise ValueError("%s must be one of %s" % (name, sorted(map(str, table))))
    return act


def _raise(st, where):
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
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return short_conv_fwd(x, weight, bias, state, cu_seqlens, activation,
                                  output_final_state, y, state_T)
    dev, index, dt = x.device, x.get_device(), x.dtype
    B, T, D, n_seq, cu = _batch(x, cu_seqlens, index, "x")
    code = _code(x)
    ld_x = _rows("x", x, x.shape, dt, index, D)
    W = _conv_width(weight, D)
    w = _required("weight", weight, (D, W), _F32, index)
    b = _dense("bias", bias, (D,), _F32, index)
    s0 = _dense("state", state, (n_seq, W - 1, D), dt, index)
    act = _act(_CONV_ACT, "activation", activation)
    y = _new(y, "y", (B, T, D), dt, dev, index)
    if output_final_state or state_T is not None:
        state_T = _new(state_T, "state_T", (n_seq, W - 1, D), dt, dev, index)
    st = _m.lib().mdn_short_conv_fwd(x.data_ptr(), w, b, s0, y.data_ptr(), _address(state_T), cu,
                                     n_seq, B, T, D, W, act, ld_x, code, _handle(index))
    if st:
        _raise(st, "mdn_short_conv_fwd")
    return y, state_T


def _conv_width(weight, D):
    if weight is None or weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError("weight must be [D, width]")
    return weight.shape[1]


def short_conv_bwd(x, weight, dy, bias=None, state=None, cu_seqlens=None, activation="silu",
                   dstate_T=None, need_dstate=None, workspace=None, stream=None):
    """Gradient of ``short_conv_fwd`` (``mdn_short_conv_bwd``) from its inputs,
    the adjoint dy of y and optionally ``dstate_T`` of the final state.
    Returns a dict with dx, dw, dbias (None without a bias) and dstate (None
    unless ``need_dstate``, by default where a state was given)."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return short_conv_bwd(x, weight, dy, bias, state, cu_seqlens, activation, dstate_T,
                                  need_dstate, workspace)
    dev, index, dt = x.device, x.get_device(), x.dtype
    B, T, D, n_seq, cu = _batch(x, cu_seqlens, index, "x")
    code = _code(x)
    ld_x = _rows("x", x, x.shape, dt, index, D)
    ld_dy = _rows("dy", dy, x.shape, dt, index, D)
    W = _conv_width(weight, D)
    w = _required("weight", weight, (D, W), _F32, index)
    b = _dense("bias", bias, (D,), _F32, index)
    s0 = _dense("state", state, (n_seq, W - 1, D), dt, index)
    dsT = _dense("dstate_T", dstate_T, (n_seq, W - 1, D), dt, index)
    act = _act(_CONV_ACT, "activation", activation)
    if need_dstate is None:
        need_dstate = state is not None
    dx = torch.empty((B, T, D), dtype=dt, device=dev)
    dw = torch.empty_like(weight)
    dbias = torch.empty_like(bias) if bias is not None else None
    dstate = torch.empty((n_seq, W - 1, D), dtype=dt, device=dev) if need_dstate else None
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_short_conv_bwd_workspace_size", B * T, D, W, code), dev, index)
    st = _m.lib().mdn_short_conv_bwd(
        x.data_ptr(), w, b, s0, dy.data_ptr(), dsT, dx.data_ptr(), dw.data_ptr(), _address(dbias),
        _address(dstate), cu, n_seq, B, T, D, W, act, ld_x, ld_dy, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_short_conv_bwd")
    return {"dx": dx, "dw": dw, "dbias": dbias, "dstate": dstate}


def short_conv_step(x, weight, state, bias=None, activation="silu", state_out=None, y=None,
                    stream=None):
    """One new token per sequence (``mdn_short_conv_step``): x ``[N, D]``, state
    ``[N, width - 1, D]``, shifted by the token in place or into ``state_out``.
    Returns y ``[N, D]``."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return short_conv_step(x, weight, state, bias, activation, state_out, y)
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    N, D = x.shape
    dev, index, dt = x.device, x.get_device(), x.dtype
    code = _code(x)
    ld_x = _rows("x", x, x.shape, dt, index, D)
    W = _conv_width(weight, D)
    w = _required("weight", weight, (D, W), _F32, index)
    b = _dense("bias", bias, (D,), _F32, index)
    s0 = _required("state", state, (N, W - 1, D), dt, index)
    so = s0 if state_out is None else _dense("state_out", state_out, (N, W - 1, D), dt, index)
    act = _act(_CONV_ACT, "activation", activation)
    y = _new(y, "y", (N, D), dt, dev, index)
    st = _m.lib().mdn_short_conv_step(x.data_ptr(), w, b, s0, so, y.data_ptr(), N, D, W, act, ld_x,
                                      code, _handle(index))
    if st:
        _raise(st, "mdn_short_conv_step")
    return y


# ------------------------------------------------------------------- scan

def ssm_state_slots(n_seq, B, T, packed):
    """Slots of the saved states (``mdn_ssm_state_slots``): chunk c of 32 tokens
    of sequence s at slot s * ceil(T / 32) + c, or, packed, at
    sum_{s' < s} ceil(L_s' / 32) + c."""
    return int(_m.lib().mdn_ssm_state_slots(int(n_seq), int(B), int(T), 1 if packed else 0))


def _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, index, D):
    """Checks the tensors every form of the scan takes; (G, N, addresses of u ..
    Cm, of D_skip, z and dt_bias, row strides)."""
    shape, dtype = u.shape, u.dtype
    if Bm is None or Bm.dim() != len(shape) + 1:
        raise ValueError("Bm must be [..., G, N]")
    bc = Bm.shape
    G, N = bc[-2:]
    if bc[:-2] != shape[:-1]:
        raise ValueError("Bm has shape %s, expected %s" % (tuple(bc), tuple(shape[:-1]) + (G, N)))
    lds = (_rows("u", u, shape, dtype, index, D), _rows("dt", dt, shape, dtype, index, D),
           _rows("Bm", Bm, bc, dtype, index, G * N, 2), _rows("Cm", Cm, bc, dtype, index, G * N, 2),
           _rows("z", z, shape, dtype, index, D) if z is not None else 0)
    ptrs = (u.data_ptr(), dt.data_ptr(), _required("A", A, (D, N), _F32, index), Bm.data_ptr(),
            Cm.data_ptr(), _dense("D_skip", D_skip, (D,), _F32, index), _address(z),
            _dense("dt_bias", dt_bias, (D,), _F32, index))
    return G, N, ptrs, lds


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
    if _elsewhere(u, "u", stream):
        with _on(u, stream):
            return ssm_scan_fwd(u, dt, A, Bm, Cm, D_skip, z, dt_bias, softplus, h0, cu_seqlens,
                                output_final_state, return_chunk_states, y, h_T, workspace)
    dev, index, dtype = u.device, u.get_device(), u.dtype
    B, T, D, n_seq, cu = _batch(u, cu_seqlens, index, "u")
    code = _code(u)
    G, N, ptrs, lds = _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, index, D)
    s0 = _dense("h0", h0, (n_seq, D, N), _F32, index)
    y = _new(y, "y", (B, T, D), dtype, dev, index)
    if output_final_state or h_T is not None:
        h_T = _new(h_T, "h_T", (n_seq, D, N), _F32, dev, index)
    h_chunks = None
    if return_chunk_states:
        slots = _size("mdn_ssm_state_slots", n_seq, B, T, cu is not None)
        h_chunks = torch.empty((slots, D, N), dtype=_F32, device=dev)
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_ssm_scan_fwd_workspace_size", n_seq, B * T, D, G, N, code), dev, index)
    st = _m.lib().mdn_ssm_scan_fwd(
        *ptrs, s0, y.data_ptr(), _address(h_T), _address(h_chunks), cu, n_seq, B, T, D, G, N,
        1 if softplus else 0, *lds, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_ssm_scan_fwd")
    return (y, h_T, h_chunks) if return_chunk_states else (y, h_T)


def ssm_scan_bwd(u, dt, A, Bm, Cm, h_chunks, dy, D_skip=None, z=None, dt_bias=None, softplus=True,
                 cu_seqlens=None, dh_T=None, need_dh0=False, workspace=None, stream=None):
    """Gradient of ``ssm_scan_fwd`` (``mdn_ssm_scan_bwd``) from its inputs, its
    chunk states (``return_chunk_states=True``), the adjoint dy of y and
    optionally ``dh_T`` of the final states.  Returns a dict with du, ddt, dA,
    dB, dC, dD_skip, dz, ddt_bias and dh0 (None where the input is None, dh0
    unless ``need_dh0``)."""
    if _elsewhere(u, "u", stream):
        with _on(u, stream):
            return ssm_scan_bwd(u, dt, A, Bm, Cm, h_chunks, dy, D_skip, z, dt_bias, softplus,
                                cu_seqlens, dh_T, need_dh0, workspace)
    dev, index, dtype = u.device, u.get_device(), u.dtype
    B, T, D, n_seq, cu = _batch(u, cu_seqlens, index, "u")
    code = _code(u)
    G, N, ptrs, lds = _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, index, D)
    ld_dy = _rows("dy", dy, u.shape, dtype, index, D)
    slots = _size("mdn_ssm_state_slots", n_seq, B, T, cu is not None)
    hc = _required("h_chunks", h_chunks, (slots, D, N), _F32, index)
    dhT = _dense("dh_T", dh_T, (n_seq, D, N), _F32, index)
    shape = (B, T, D)
    g = {"du": torch.empty(shape, dtype=dtype, device=dev),
         "ddt": torch.empty(shape, dtype=dtype, device=dev),
         "dA": torch.empty_like(A),
         "dB": torch.empty((B, T, G, N), dtype=dtype, device=dev),
         "dC": torch.empty((B, T, G, N), dtype=dtype, device=dev),
         "dD_skip": torch.empty_like(D_skip) if D_skip is not None else None,
         "dz": torch.empty(shape, dtype=dtype, device=dev) if z is not None else None,
         "ddt_bias": torch.empty_like(dt_bias) if dt_bias is not None else None,
         "dh0": torch.empty((n_seq, D, N), dtype=_F32, device=dev) if need_dh0 else None}
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_ssm_scan_bwd_workspace_size", n_seq, B * T, D, G, N, code), dev, index)
    st = _m.lib().mdn_ssm_scan_bwd(
        *ptrs, hc, dy.data_ptr(), dhT, *map(_address, g.values()), cu, n_seq, B, T, D, G, N,
        1 if softplus else 0, *lds, ld_dy, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_ssm_scan_bwd")
    return g


def ssm_scan_step(u, dt, A, Bm, Cm, h, D_skip=None, z=None, dt_bias=None, softplus=True,
                  h_out=None, y=None, stream=None):
    """One token per sequence (``mdn_ssm_scan_step``): u, dt, z ``[N, D]``, Bm, Cm
    ``[N, G, n_states]``; h ``[N, D, n_states]`` fp32 is updated in place or
    into ``h_out``.  Returns y ``[N, D]``."""
    if _elsewhere(u, "u", stream):
        with _on(u, stream):
            return ssm_scan_step(u, dt, A, Bm, Cm, h, D_skip, z, dt_bias, softplus, h_out, y)
    if u.dim() != 2:
        raise ValueError("u must be [N, D]")
    n, D = u.shape
    dev, index = u.device, u.get_device()
    code = _code(u)
    G, N, ptrs, lds = _scan_inputs(u, dt, A, Bm, Cm, D_skip, z, dt_bias, index, D)
    s0 = _required("h", h, (n, D, N), _F32, index)
    so = s0 if h_out is None else _dense("h_out", h_out, (n, D, N), _F32, index)
    y = _new(y, "y", (n, D), u.dtype, dev, index)
    st = _m.lib().mdn_ssm_scan_step(*ptrs, s0, so, y.data_ptr(), n, D, G, N, 1 if softplus else 0,
                                    *lds, code, _handle(index))
    if st:
        _raise(st, "mdn_ssm_scan_step")
    return y


# ------------------------------------------------------------------ norms

def _norm_inputs(y, x, gate, w_post, w_pre, scale, gate_act, index):
    """Checks what both directions take; (D, rows, addresses, row strides, act)."""
    shape, dtype = y.shape, y.dtype
    if y.dim() < 1 or shape[-1] == 0:
        raise ValueError("y must be [..., D] with at least one column")
    D = shape[-1]
    if y.numel() > 0x7fffffff * D:
        raise ValueError("y has more than 2^31 - 1 rows")
    lds = (_rows("y", y, shape, dtype, index, D), _rows("x", x, shape, dtype, index, D),
           _rows("gate", gate, shape, dtype, index, D) if gate is not None else 0)
    ptrs = (y.data_ptr(), x.data_ptr(), _address(gate), _dense("w_post", w_post, (D,), _F32, index),
            _dense("w_pre", w_pre, (D,), _F32, index), _dense("scale", scale, (D,), _F32, index))
    return D, y.numel() // D, ptrs, lds, _act(_GATE_ACT, "gate_act", gate_act)


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
    if _elsewhere(y, "y", stream):
        with _on(y, stream):
            return norm_residual_fwd(y, x, w_post, w_pre, gate, gate_act, scale, eps, return_stats,
                                     x_out)
    dev, index, dtype, shape = y.device, y.get_device(), y.dtype, y.shape
    code = _code(y)
    D, rows, ptrs, lds, act = _norm_inputs(y, x, gate, w_post, w_pre, scale, gate_act, index)
    x_out = _new(x_out, "x_out", shape, dtype, dev, index)
    h = torch.empty(shape, dtype=dtype, device=dev) if w_pre is not None else None
    stats = torch.empty(shape[:-1] + (2,), dtype=_F32, device=dev) if return_stats else None
    st = _m.lib().mdn_norm_residual_fwd(*ptrs, x_out.data_ptr(), _address(h), _address(stats), rows,
                                        D, act, eps, *lds, code, _handle(index))
    if st:
        _raise(st, "mdn_norm_residual_fwd")
    return (x_out, h, stats) if return_stats else (x_out, h)


def norm_residual_bwd(y, x, stats, dx_out, dh=None, w_post=None, w_pre=None, gate=None,
                      gate_act="sigmoid", scale=None, eps=1e-6, workspace=None, stream=None):
    """Gradient of ``norm_residual_fwd`` (``mdn_norm_residual_bwd``) from its
    inputs, its stats and the adjoints of x_out and h.  ``eps`` is accepted for
    symmetry; the stats already hold it.  Returns a dict with dy, dx, dgate,
    dw_post, dw_pre and dscale (None where the input is None)."""
    if _elsewhere(y, "y", stream):
        with _on(y, stream):
            return norm_residual_bwd(y, x, stats, dx_out, dh, w_post, w_pre, gate, gate_act, scale,
                                     eps, workspace)
    dev, index, dtype, shape = y.device, y.get_device(), y.dtype, y.shape
    code = _code(y)
    D, rows, ptrs, lds, act = _norm_inputs(y, x, gate, w_post, w_pre, scale, gate_act, index)
    st2 = _required("stats", stats, shape[:-1] + (2,), _F32, index)
    ld_dx_out = _rows("dx_out", dx_out, shape, dtype, index, D)
    if w_pre is not None and dh is None:
        raise ValueError("dh is required with w_pre")
    ld_dh = _rows("dh", dh, shape, dtype, index, D) if dh is not None else 0
    g = {"dy": torch.empty(shape, dtype=dtype, device=dev),
         "dx": torch.empty(shape, dtype=dtype, device=dev),
         "dgate": torch.empty(shape, dtype=dtype, device=dev) if gate is not None else None,
         "dw_post": torch.empty_like(w_post) if w_post is not None else None,
         "dw_pre": torch.empty_like(w_pre) if w_pre is not None else None,
         "dscale": torch.empty_like(scale) if scale is not None else None}
    workspace, ws, nbytes = _workspace(
        workspace, _size("mdn_norm_residual_bwd_workspace_size", rows, D, code), dev, index)
    st = _m.lib().mdn_norm_residual_bwd(
        *ptrs, st2, dx_out.data_ptr(), _address(dh), *map(_address, g.values()), rows, D, act, *lds,
        ld_dx_out, ld_dh, code, ws, nbytes, _handle(index))
    if st:
        _raise(st, "mdn_norm_residual_bwd")
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
