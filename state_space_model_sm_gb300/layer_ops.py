"""The operators a layer needs around the scan: the short causal convolution,
the selective scan (a decay per channel and state), one token of each scan for
decoding, and the residual / norm step between layers.

Bindings of the same names as ``include/ssd.h`` declares (without the prefix):
they check the tensors, allocate outputs and workspace, and pass pointers and
the current stream.  Inputs are float32 or bfloat16 CUDA tensors; parameters
(weights, biases, A, D) and scan states are float32.  Tensors live on the current
device (those of another one are refused).  Every call is asynchronous and its
results are ordered on the current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native

_CODE = {torch.float32: 0, torch.bfloat16: 1}  # ssd_dtype
_F32, _I32 = torch.float32, torch.int32
_empty, _empty_like = torch.empty, torch.empty_like  # (Tensor.new_empty takes twice as long)
_stream = torch._C._cuda_getCurrentRawStream  # of a device index; no Stream object
_current_device = torch._C._cuda_getDevice
_lib = None


def _native_lib():
    global _lib
    if _lib is None:
        _lib = _native.load()
    return _lib


def _fail(fn, status):
    from . import SSDError
    raise SSDError(fn, status)


def _code(dtype):
    c = _CODE.get(dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    return c


def _device(t):
    """Index of t's device, which has to be the current one: the library launches
    there, whatever device the stream and the addresses are of."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    if dev != _current_device():
        raise ValueError(f"tensors live on cuda:{dev}, but the current device is "
                         f"cuda:{_current_device()}")
    return dev


def _lead(t, name, ndim):
    """Index of the device of the call's first tensor, whose rank is checked."""
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got {tuple(t.shape)}")
    return _device(t)


def _wrong(t, name, shape, dtype, device):
    """Raises what is wrong with t (apart from its strides)."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected device cuda:{device}, got {t.device}")


def _check(t, name, shape, dtype, device):
    """Shape, type, device and density of t; its address (None for None)."""
    if t is None:
        return None
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != device
            or not t.is_contiguous()):
        _wrong(t, name, shape, dtype, device)
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, lead, dtype, device):
    """As _check for an input that may be a column range of a wider tensor: the
    ``lead`` leading dimensions (batch, or batch and position) may be strided, the
    others are dense.  Returns (address, elements between rows, elements between
    batch rows); a row stride of 0 stands for a dense tensor."""
    if t is None:
        return None, 0, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _wrong(t, name, shape, dtype, device)
    if t.is_contiguous():
        return t.data_ptr(), 0, 0
    dense, stride = 1, t.stride()
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and stride[i] != dense:
            raise ValueError(f"{name}: columns must be contiguous")
        dense *= shape[i]
    row = stride[lead - 1] if shape[lead - 1] > 1 else dense
    if row < dense:
        raise ValueError(f"{name}: rows must not overlap")
    return t.data_ptr(), row, stride[0]


def _output(t, name, shape, dtype, like):
    """t after its check, or a new tensor, on the device of ``like``."""
    if t is None:
        return _empty(shape, dtype=dtype, device=like.device)
    _check(t, name, shape, dtype, like.get_device())
    return t


def _outputs(out, want, like):
    """The named outputs (name, shape, dtype), new or from the caller's dict."""
    if out is None:
        dev = like.device
        return {k: _empty(s, dtype=t, device=dev) for k, s, t in want}
    return {k: _output(out.get(k), k, s, t, like) for k, s, t in want}


def _scratch(nbytes, like, workspace):
    if workspace is None:
        return _empty(nbytes, dtype=torch.uint8, device=like.device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous on {like.device}")
    return workspace


def _at(t):
    return None if t is None else t.data_ptr()


# --------------------------------------------------------- causal convolution

def _conv_inputs(x, w, bias, ndim, silu, out_dtype):
    dev = _lead(x, "x", ndim)
    xshape, xd = x.shape, x.dtype
    batch, C = xshape[0], xshape[-1]
    T = xshape[1] if ndim == 3 else 1
    wshape = w.shape
    if len(wshape) != 2:
        raise ValueError("w must be (channels, width)")
    K = wshape[1]
    xp, xs, xb = _rows(x, "x", xshape, ndim - 1, xd, dev)
    wp = _check(w, "w", (C, K), _F32, dev)
    bp = None if bias is None else _check(bias, "bias", (C,), _F32, dev)
    code = _code(xd)
    if out_dtype is None:
        out_dtype, ocode = xd, code
    else:
        ocode = _code(out_dtype)
    shape = _native.ConvShape(batch, T, C, K, xs, xb, 1 if silu else 0, code, ocode)
    return dev, shape, (batch, T, C, K), out_dtype, xp, wp, bp


def causal_conv_fwd(x, w, bias=None, init_state=None, lengths=None, silu: bool = True,
                    out_dtype=None, return_final_state: bool = True, y=None, final_state=None):
    """y, final_state = the causal depthwise convolution of x over the last
    ``width`` positions, with SiLU unless ``silu=False`` (``ssd_causal_conv_fwd``).

    x (batch, seqlen, channels), may be a column range of a wider tensor; w
    (channels, width) with width 2 to 4 and bias (channels,) float32; init_state
    (batch, width - 1, channels) in x's type: the inputs before position 0;
    lengths (batch,) int32: positions from lengths[b] on are padding.
    final_state is the state after lengths[b] positions, which
    ``causal_conv_step`` goes on from (a given one must not overlap init_state).  y is in ``out_dtype`` (x's type)."""
    lib = _native_lib()
    dev, shape, (B, T, C, K), odt, xp, wp, bp = _conv_inputs(x, w, bias, 3, silu, out_dtype)
    ip = _check(init_state, "init_state", (B, K - 1, C), x.dtype, dev)
    lp = _check(lengths, "lengths", (B,), _I32, dev)
    y = _output(y, "y", (B, T, C), odt, x)
    if return_final_state:
        final_state = _output(final_state, "final_state", (B, K - 1, C), x.dtype, x)
    else:
        final_state = None
    st = lib.ssd_causal_conv_fwd(shape, xp, wp, bp, ip, lp, y.data_ptr(), _at(final_state),
                                 _stream(dev))
    if st:
        _fail("ssd_causal_conv_fwd", st)
    return y, final_state


def causal_conv_bwd(x, w, bias, dy, init_state=None, lengths=None, silu: bool = True,
                    dfinal_state=None, out_dtype=None, workspace=None, out=None):
    """Gradients of <dy, y> + <dfinal_state, final_state> of ``causal_conv_fwd``
    (``ssd_causal_conv_bwd``): a dict with dx (``out_dtype``, x's type by default),
    dw and dbias (float32) and, with init_state, dinit_state (``out_dtype``)."""
    lib = _native_lib()
    dev, shape, (B, T, C, K), odt, xp, wp, bp = _conv_inputs(x, w, bias, 3, silu, out_dtype)
    ip = _check(init_state, "init_state", (B, K - 1, C), x.dtype, dev)
    lp = _check(lengths, "lengths", (B,), _I32, dev)
    gp = _check(dy, "dy", (B, T, C), x.dtype, dev)
    fp = _check(dfinal_state, "dfinal_state", (B, K - 1, C), x.dtype, dev)
    want = [("dx", (B, T, C), odt), ("dw", (C, K), _F32), ("dbias", (C,), _F32)]
    if init_state is not None:
        want.append(("dinit_state", (B, K - 1, C), odt))
    out = _outputs(out, want, x)
    nbytes = lib.ssd_causal_conv_workspace_size(shape)
    ws = _scratch(max(nbytes, 1), x, workspace)
    st = lib.ssd_causal_conv_bwd(shape, xp, wp, bp, ip, lp, gp, fp, out["dx"].data_ptr(),
                                 out["dw"].data_ptr(), out["dbias"].data_ptr(),
                                 _at(out.get("dinit_state")), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_causal_conv_bwd", st)
    return out


# The decoding calls (one token, and the block norm between layers) take a few
# microseconds on the GPU, so their checks are written out in one condition for
# the plain case (dense tensors, the default output); anything else goes through
# the checks of the helpers above, which also say what is wrong.

def causal_conv_step(x, state, w, bias=None, slots=None, silu: bool = True, out_dtype=None, y=None):
    """One token of ``causal_conv_fwd`` (``ssd_causal_conv_step``): x, y (batch,
    channels); state (nslots, width - 1, channels) in x's type, updated in place.
    slots (batch,) int32 names each row's state; a negative one marks an empty
    row, whose output is 0."""
    lib, xs, ws, ss, xd, dev = _lib, x.shape, w.shape, state.shape, x.dtype, x.get_device()
    if (lib is not None and dev >= 0 and dev == _current_device()
            and len(xs) == 2 and len(ws) == 2 and xd in _CODE
            and out_dtype is None and y is None and x.is_contiguous()
            and ws[0] == xs[1] and w.dtype is _F32 and w.get_device() == dev and w.is_contiguous()
            and ss == (ss[0], ws[1] - 1, xs[1]) and state.dtype is xd
            and state.get_device() == dev and state.is_contiguous()
            and (bias is None or (bias.shape == xs[1:] and bias.dtype is _F32
                                  and bias.get_device() == dev and bias.is_contiguous()))
            and (slots is None or (slots.shape == xs[:1] and slots.dtype is _I32
                                   and slots.get_device() == dev and slots.is_contiguous()))):
        code = _CODE[xd]
        shape = _native.ConvShape(xs[0], 1, xs[1], ws[1], 0, 0, 1 if silu else 0, code, code)
        y = _empty_like(x)
        st = lib.ssd_causal_conv_step(
            shape, x.data_ptr(), state.data_ptr(), w.data_ptr(),
            None if bias is None else bias.data_ptr(), None if slots is None else slots.data_ptr(),
            ss[0], y.data_ptr(), _stream(dev))
    else:
        lib = _native_lib()
        dev, shape, (B, _, C, K), odt, xp, wp, bp = _conv_inputs(x, w, bias, 2, silu, out_dtype)
        sp = _check(state, "state", (state.shape[0], K - 1, C), x.dtype, dev)
        lp = _check(slots, "slots", (B,), _I32, dev)
        y = _output(y, "y", (B, C), odt, x)
        st = lib.ssd_causal_conv_step(shape, xp, sp, wp, bp, lp, state.shape[0], y.data_ptr(),
                                      _stream(dev))
    if st:
        _fail("ssd_causal_conv_step", st)
    return y


# ------------------------------------------------------------- selective scan

def _sel_inputs(x, dt, dt_bias, A, B, C, D, z, ndim, out_dtype):
    dev = _lead(x, "x", ndim)
    xshape, xd = x.shape, x.dtype
    if B.dim() != ndim + 1 or A.dim() != 2:
        raise ValueError("A must be (channels, dstate), B and C (..., ngroups, dstate)")
    batch, ch = xshape[0], xshape[-1]
    T = xshape[1] if ndim == 3 else 1
    N, G = A.shape[1], B.shape[-2]
    gn = (batch, T, G, N) if ndim == 3 else (batch, G, N)
    lead = ndim - 1
    bp, bs, bb = _rows(B, "B", gn, lead, xd, dev)
    cp, cs, cb = _rows(C, "C", gn, lead, xd, dev)
    zp, zs, zb = (None, 0, 0) if z is None else _rows(z, "z", xshape, lead, xd, dev)
    ptrs = (_check(x, "x", xshape, xd, dev), _check(dt, "dt", xshape, xd, dev),
            _check(dt_bias, "dt_bias", (ch,), _F32, dev), _check(A, "A", (ch, N), _F32, dev),
            bp, cp, _check(D, "D", (ch,), _F32, dev), zp)
    code = _code(xd)
    if out_dtype is None:
        out_dtype, ocode = xd, code
    else:
        ocode = _code(out_dtype)
    shape = _native.SelectiveShape(batch, T, ch, N, G, zs, bs, cs, zb, bb, cb, code, ocode)
    return dev, shape, (batch, T, ch, N, G), out_dtype, ptrs


def selective_scan_fwd(x, dt, dt_bias, A, B, C, D=None, z=None, init_states=None, lengths=None,
                       out_dtype=None, return_final_states: bool = True, workspace=None, out=None,
                       final_states=None):
    """out, final_states = the selective scan of x (``ssd_selective_scan_fwd``):
    h <- exp(delta A) h + delta x B with delta = softplus(dt + dt_bias) per channel,
    y = C . h + D x, times silu(z) when z is given.

    x, dt, z (batch, seqlen, channels); B, C (batch, seqlen, ngroups, dstate) (z, B
    and C may be column ranges of wider tensors); A (channels, dstate), dt_bias and D
    (channels,), init_states (batch, channels, dstate) float32; lengths (batch,)
    int32: positions from lengths[b] on are padding.  dstate <= 64.  final_states
    is what ``selective_step`` goes on from."""
    lib = _native_lib()
    dev, shape, (Bt, T, ch, N, G), odt, p = _sel_inputs(x, dt, dt_bias, A, B, C, D, z, 3, out_dtype)
    ip = _check(init_states, "init_states", (Bt, ch, N), _F32, dev)
    lp = _check(lengths, "lengths", (Bt,), _I32, dev)
    out = _output(out, "out", (Bt, T, ch), odt, x)
    if return_final_states:
        final_states = _output(final_states, "final_states", (Bt, ch, N), _F32, x)
    else:
        final_states = None
    nbytes = lib.ssd_selective_scan_fwd_workspace_size(shape)
    ws = _scratch(max(nbytes, 1), x, workspace)
    st = lib.ssd_selective_scan_fwd(shape, *p, ip, lp, out.data_ptr(), _at(final_states),
                                    ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_selective_scan_fwd", st)
    return out, final_states


def selective_scan_bwd(x, dt, dt_bias, A, B, C, D, z, dout, init_states=None, lengths=None,
                       dfinal_states=None, out_dtype=None, workspace=None, out=None):
    """Gradients of <dout, out> + <dfinal_states, final_states> of
    ``selective_scan_fwd`` (``ssd_selective_scan_bwd``): a dict with dx, ddt and,
    with z, dz in ``out_dtype`` (x's type), and dA, dB, dC, dD, ddt_bias and, with
    init_states, dinit_states in float32."""
    lib = _native_lib()
    dev, shape, (Bt, T, ch, N, G), odt, p = _sel_inputs(x, dt, dt_bias, A, B, C, D, z, 3, out_dtype)
    ip = _check(init_states, "init_states", (Bt, ch, N), _F32, dev)
    lp = _check(lengths, "lengths", (Bt,), _I32, dev)
    gp = _check(dout, "dout", (Bt, T, ch), x.dtype, dev)
    fp = _check(dfinal_states, "dfinal_states", (Bt, ch, N), _F32, dev)
    want = [("dx", (Bt, T, ch), odt), ("ddt", (Bt, T, ch), odt), ("dA", (ch, N), _F32),
            ("dB", (Bt, T, G, N), _F32), ("dC", (Bt, T, G, N), _F32), ("dD", (ch,), _F32),
            ("ddt_bias", (ch,), _F32)]
    if z is not None:
        want.append(("dz", (Bt, T, ch), odt))
    if init_states is not None:
        want.append(("dinit_states", (Bt, ch, N), _F32))
    out = _outputs(out, want, x)
    nbytes = lib.ssd_selective_scan_bwd_workspace_size(shape)
    ws = _scratch(max(nbytes, 1), x, workspace)
    st = lib.ssd_selective_scan_bwd(
        shape, *p, ip, lp, gp, fp, *(_at(out.get(k)) for k in (
            "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit_states")),
        ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_selective_scan_bwd", st)
    return out


def selective_step(x, dt, dt_bias, A, B, C, state, D=None, z=None, slots=None, out_dtype=None, y=None):
    """One token of ``selective_scan_fwd`` (``ssd_selective_step``): x, dt, z, y
    (batch, channels); B, C (batch, ngroups, dstate); state (nslots, channels,
    dstate) float32, updated in place; slots as in ``causal_conv_step``."""
    lib, xs, bs, ss, xd, dev = _lib, x.shape, B.shape, state.shape, x.dtype, x.get_device()
    if (lib is not None and dev >= 0 and dev == _current_device()
            and len(xs) == 2 and len(bs) == 3 and xd in _CODE
            and out_dtype is None and y is None and x.is_contiguous()
            and dt.shape == xs and dt.dtype is xd and dt.get_device() == dev and dt.is_contiguous()
            and bs[0] == xs[0] and B.dtype is xd and B.get_device() == dev and B.is_contiguous()
            and C.shape == bs and C.dtype is xd and C.get_device() == dev and C.is_contiguous()
            and ss == (ss[0], xs[1], bs[2]) and state.dtype is _F32
            and state.get_device() == dev and state.is_contiguous()
            and A.shape == ss[1:] and A.dtype is _F32 and A.get_device() == dev
            and A.is_contiguous()
            and (z is None or (z.shape == xs and z.dtype is xd and z.get_device() == dev
                               and z.is_contiguous()))
            and (dt_bias is None or (dt_bias.shape == xs[1:] and dt_bias.dtype is _F32
                                     and dt_bias.get_device() == dev and dt_bias.is_contiguous()))
            and (D is None or (D.shape == xs[1:] and D.dtype is _F32 and D.get_device() == dev
                               and D.is_contiguous()))
            and (slots is None or (slots.shape == xs[:1] and slots.dtype is _I32
                                   and slots.get_device() == dev and slots.is_contiguous()))):
        code = _CODE[xd]
        shape = _native.SelectiveShape(xs[0], 1, xs[1], bs[2], bs[1], 0, 0, 0, 0, 0, 0, code, code)
        y = _empty_like(x)
        st = lib.ssd_selective_step(
            shape, x.data_ptr(), dt.data_ptr(), None if dt_bias is None else dt_bias.data_ptr(),
            A.data_ptr(), B.data_ptr(), C.data_ptr(), None if D is None else D.data_ptr(),
            None if z is None else z.data_ptr(), state.data_ptr(),
            None if slots is None else slots.data_ptr(), ss[0], y.data_ptr(), _stream(dev))
    else:
        lib = _native_lib()
        dev, shape, (Bt, _, ch, N, G), odt, p = _sel_inputs(x, dt, dt_bias, A, B, C, D, z, 2,
                                                            out_dtype)
        sp = _check(state, "state", (state.shape[0], ch, N), _F32, dev)
        lp = _check(slots, "slots", (Bt,), _I32, dev)
        y = _output(y, "y", (Bt, ch), odt, x)
        st = lib.ssd_selective_step(shape, *p, sp, lp, state.shape[0], y.data_ptr(), _stream(dev))
    if st:
        _fail("ssd_selective_step", st)
    return y


def ssd_step(x, dt, dt_bias, A, B, C, state, D=None, slots=None, out_dtype=None, y=None):
    """One token of ``ssd_fwd``'s scan (``ssd_step``): x, y (batch, nheads, headdim),
    dt (batch, nheads), B, C (batch, ngroups, dstate); A, dt_bias, D (nheads,) and
    state (nslots, nheads, headdim, dstate) float32, the state updated in place;
    slots as in ``causal_conv_step``.  y is in ``out_dtype`` (x's type)."""
    lib, xs, bs, ss, xd, dev = _lib, x.shape, B.shape, state.shape, x.dtype, x.get_device()
    if (lib is not None and dev >= 0 and dev == _current_device()
            and len(xs) == 3 and len(bs) == 3 and xd in _CODE
            and out_dtype is None and y is None and x.is_contiguous()
            and dt.shape == xs[:2] and dt.dtype is xd and dt.get_device() == dev
            and dt.is_contiguous()
            and bs[0] == xs[0] and B.dtype is xd and B.get_device() == dev and B.is_contiguous()
            and C.shape == bs and C.dtype is xd and C.get_device() == dev and C.is_contiguous()
            and ss == (ss[0], xs[1], xs[2], bs[2]) and state.dtype is _F32
            and state.get_device() == dev and state.is_contiguous()
            and A.shape == xs[1:2] and A.dtype is _F32 and A.get_device() == dev
            and A.is_contiguous()
            and (dt_bias is None or (dt_bias.shape == xs[1:2] and dt_bias.dtype is _F32
                                     and dt_bias.get_device() == dev and dt_bias.is_contiguous()))
            and (D is None or (D.shape == xs[1:2] and D.dtype is _F32 and D.get_device() == dev
                               and D.is_contiguous()))
            and (slots is None or (slots.shape == xs[:1] and slots.dtype is _I32
                                   and slots.get_device() == dev and slots.is_contiguous()))):
        code = _CODE[xd]
        shape = _native.Shape(xs[0], 1, xs[1], xs[2], bs[2], bs[1], 1, code, code)
        y = _empty_like(x)
        st = lib.ssd_step(
            shape, x.data_ptr(), dt.data_ptr(), None if dt_bias is None else dt_bias.data_ptr(),
            A.data_ptr(), B.data_ptr(), C.data_ptr(), None if D is None else D.data_ptr(),
            state.data_ptr(), None if slots is None else slots.data_ptr(), ss[0], y.data_ptr(),
            _stream(dev))
    else:
        lib = _native_lib()
        dev = _lead(x, "x", 3)
        if B.dim() != 3:
            raise ValueError("B and C must be (batch, ngroups, dstate)")
        Bt, H, P = x.shape
        G, N = B.shape[1:]
        odt = xd if out_dtype is None else out_dtype
        shape = _native.Shape(Bt, 1, H, P, N, G, 1, _code(xd), _code(odt))
        p = (_check(x, "x", x.shape, xd, dev), _check(dt, "dt", (Bt, H), xd, dev),
             _check(dt_bias, "dt_bias", (H,), _F32, dev), _check(A, "A", (H,), _F32, dev),
             _check(B, "B", (Bt, G, N), xd, dev), _check(C, "C", (Bt, G, N), xd, dev),
             _check(D, "D", (H,), _F32, dev),
             _check(state, "state", (state.shape[0], H, P, N), _F32, dev),
             _check(slots, "slots", (Bt,), _I32, dev))
        y = _output(y, "y", (Bt, H, P), odt, x)
        st = lib.ssd_step(shape, *p, state.shape[0], y.data_ptr(), _stream(dev))
    if st:
        _fail("ssd_step", st)
    return y


# ------------------------------------------------------------------ block norm

def _bn_inputs(residual, o, w_pre, w_post, gate, scale, eps):
    rshape = residual.shape
    if len(rshape) < 1:
        raise ValueError("residual must be a CUDA tensor (..., features)")
    dev = _device(residual)
    F = rshape[-1]
    rows = residual.numel() // F if F else 0
    rd, od, ng, gp = residual.dtype, o.dtype, 0, None
    if gate is not None:
        ng = gate.numel() // F if F else 0
        gp = _check(gate, "gate", (ng, F), _F32, dev)
        if ng < 1 or rows % ng != 0:
            raise ValueError(f"gate: {ng} gate rows do not divide {rows} rows")
    ptrs = (_check(residual, "residual", rshape, rd, dev), _check(o, "o", rshape, od, dev),
            _check(w_pre, "w_pre", (F,), _F32, dev), _check(w_post, "w_post", (F,), _F32, dev), gp)
    shape = _native.BlockNormShape(rows, F, ng, eps, scale, _code(od), _code(rd))
    return dev, shape, F, ptrs


def block_norm_fwd(residual, o, w_pre, w_post=None, gate=None, scale: float = 1.0,
                   eps: float = 1e-5, residual_out=None, h=None):
    """residual_out, h of the step between two layers (``ssd_block_norm_fwd``):
    residual_out = residual + scale * gate * t, with t = rmsnorm(o) * w_post (o itself
    without w_post), and h = rmsnorm(residual_out) * w_pre, the next layer's input.

    residual (..., features) float32 or bfloat16; o of its shape, bfloat16 or
    float32 (float32 needs a float32 residual); w_pre, w_post (features,) float32;
    gate (ngates, features) float32: one row for all, one per sequence or one per
    row, each covering rows / ngates consecutive rows.  residual_out may be
    ``residual`` and h may be ``o`` (in place)."""
    lib, rs, rd, od, dev = _lib, residual.shape, residual.dtype, o.dtype, residual.get_device()
    n = len(rs)
    if (lib is not None and dev >= 0 and dev == _current_device() and n > 0 and rs[-1] > 0
            and rd in _CODE and od in _CODE
            and residual.is_contiguous() and residual_out is None and h is None
            and o.shape == rs and o.get_device() == dev and o.is_contiguous()
            and w_pre.shape == rs[n - 1:] and w_pre.dtype is _F32 and w_pre.get_device() == dev
            and w_pre.is_contiguous()
            and (w_post is None or (w_post.shape == rs[n - 1:] and w_post.dtype is _F32
                                    and w_post.get_device() == dev and w_post.is_contiguous()))
            and (gate is None or (gate.shape == (1, rs[-1]) and gate.dtype is _F32
                                  and gate.get_device() == dev and gate.is_contiguous()))):
        F = rs[-1]
        shape = _native.BlockNormShape(residual.numel() // F, F, 0 if gate is None else 1, eps,
                                       scale, _CODE[od], _CODE[rd])
        residual_out, h = _empty_like(residual), _empty_like(o)
        st = lib.ssd_block_norm_fwd(
            shape, residual.data_ptr(), o.data_ptr(), w_pre.data_ptr(),
            None if w_post is None else w_post.data_ptr(),
            None if gate is None else gate.data_ptr(), residual_out.data_ptr(), h.data_ptr(),
            _stream(dev))
    else:
        lib = _native_lib()
        dev, shape, F, p = _bn_inputs(residual, o, w_pre, w_post, gate, scale, eps)
        residual_out = _output(residual_out, "residual_out", rs, rd, residual)
        h = _output(h, "h", o.shape, od, residual)
        st = lib.ssd_block_norm_fwd(shape, *p, residual_out.data_ptr(), h.data_ptr(), _stream(dev))
    if st:
        _fail("ssd_block_norm_fwd", st)
    return residual_out, h


def block_norm_bwd(residual, o, w_pre, w_post, gate, dh, dresidual_out=None, scale: float = 1.0,
                   eps: float = 1e-5, workspace=None, out=None):
    """Gradients of <dh, h> + <dresidual_out, residual_out> of ``block_norm_fwd``
    from its inputs (``ssd_block_norm_bwd``): a dict with dresidual (residual's type),
    do (o's type), dw_pre and, with w_post and gate, dw_post and dgate (float32)."""
    lib = _native_lib()
    dev, shape, F, p = _bn_inputs(residual, o, w_pre, w_post, gate, scale, eps)
    hp = _check(dh, "dh", o.shape, o.dtype, dev)
    rp = _check(dresidual_out, "dresidual_out", residual.shape, residual.dtype, dev)
    given = out
    if given is None:
        out = {"dresidual": _empty_like(residual), "do": _empty_like(o), "dw_pre": _empty_like(w_pre)}
        if w_post is not None:
            out["dw_post"] = _empty_like(w_post)
        if gate is not None:
            out["dgate"] = _empty_like(gate)
    else:
        want = [("dresidual", residual.shape, residual.dtype), ("do", o.shape, o.dtype),
                ("dw_pre", (F,), _F32), ("dw_post", (F,), _F32)]
        out = _outputs(given, want if w_post is not None else want[:3], residual)
        if gate is not None:
            out["dgate"] = _output(given.get("dgate"), "dgate", gate.shape, _F32, residual)
    nbytes = lib.ssd_block_norm_workspace_size(shape)
    ws = _scratch(nbytes or 1, residual, workspace)
    st = lib.ssd_block_norm_bwd(
        shape, *p, hp, rp, out["dresidual"].data_ptr(), out["do"].data_ptr(),
        out["dw_pre"].data_ptr(), None if w_post is None else out["dw_post"].data_ptr(),
        None if gate is None else out["dgate"].data_ptr(), ws.data_ptr(),
        nbytes if workspace is None else ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_block_norm_bwd", st)
    return out
