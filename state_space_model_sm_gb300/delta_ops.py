"""The gated delta rule (chunked forward and backward, one token) and the norm of
queries and keys with the rotation of positions in front of it.

Bindings of the same names as ``include/ssd.h`` declares (without the prefix), in the
manner of ``layer_ops``: tensors are checked, outputs and workspace allocated, pointers
and the current stream passed on.
"""
from __future__ import annotations

from . import _native
from .layer_ops import (_CODE, _F32, _I32, _at, _check, _code, _current_device, _device, _empty,
                        _empty_like, _fail, _native_lib, _output, _outputs, _rows, _scratch, _stream)


# ---------------------------------------------------------- gated delta rule

def _delta_inputs(q, k, v, dt, dt_bias, A, beta, ndim, scale, out_dtype):
    if v.dim() != ndim or q.dim() != ndim:
        raise ValueError("q, k must be (..., ngroups, dstate) and v (..., nheads, headdim), with "
                         f"{ndim} dimensions")
    dev = _device(v)
    vs, xd = v.shape, v.dtype
    batch, H, P = vs[0], vs[-2], vs[-1]
    T = vs[1] if ndim == 4 else 1
    G, N = q.shape[-2:]
    lead = ndim - 2
    gn, ht = vs[:lead] + (G, N), vs[:lead] + (H,)
    qp, qs, qb = _rows(q, "q", gn, lead, xd, dev)
    kp, ks, kb = _rows(k, "k", gn, lead, xd, dev)
    vp, vr, vb = _rows(v, "v", vs, lead, xd, dev)
    ptrs = (qp, kp, vp, _check(dt, "dt", ht, xd, dev), _check(dt_bias, "dt_bias", (H,), _F32, dev),
            _check(A, "A", (H,), _F32, dev), _check(beta, "beta", ht, xd, dev))
    code = _code(xd)
    if out_dtype is None:
        out_dtype, ocode = xd, code
    else:
        ocode = _code(out_dtype)
    shape = _native.DeltaShape(batch, T, H, P, N, G, qs, ks, vr, qb, kb, vb, scale, code, ocode)
    return dev, shape, (batch, T, H, P, N, G), out_dtype, ptrs


def gated_delta_fwd(q, k, v, dt, dt_bias, A, beta, init_states=None, lengths=None,
                    scale: float = 1.0, out_dtype=None, return_final_states: bool = True,
                    workspace=None, y=None, final_states=None):
    """y, final_states = the gated delta rule (``ssd_gated_delta_fwd``): a state S per head
    with S <- a S, S <- S + b (v - S k) k^T, y = scale S q, where
    a = exp(softplus(dt + dt_bias) A) and b = sigmoid(beta).

    q, k (batch, seqlen, ngroups, dstate), shared by the nheads / ngroups heads of a group;
    v (batch, seqlen, nheads, headdim) (q, k and v may be column ranges of wider tensors);
    dt, beta (batch, seqlen, nheads); dt_bias (or None), A (nheads,), init_states (batch,
    nheads, headdim, dstate) float32; lengths (batch,) int32: positions from lengths[b] on
    are padding.  dstate <= 128, headdim <= 256.  Keys longer than 1 let the state grow;
    ``qk_norm_fwd(..., l2=True)`` makes unit keys.  y is in ``out_dtype`` (v's type).
    final_states is what ``gated_delta_step`` goes on from (a given one must not overlap
    init_states)."""
    lib = _native_lib()
    dev, shape, (B, T, H, P, N, G), odt, p = _delta_inputs(q, k, v, dt, dt_bias, A, beta, 4, scale,
                                                           out_dtype)
    ip = _check(init_states, "init_states", (B, H, P, N), _F32, dev)
    lp = _check(lengths, "lengths", (B,), _I32, dev)
    y = _output(y, "y", (B, T, H, P), odt, v)
    if return_final_states:
        final_states = _output(final_states, "final_states", (B, H, P, N), _F32, v)
    else:
        final_states = None
    ws = _scratch(max(lib.ssd_gated_delta_fwd_workspace_size(shape), 1), v, workspace)
    st = lib.ssd_gated_delta_fwd(shape, *p, ip, lp, y.data_ptr(), _at(final_states), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_gated_delta_fwd", st)
    return y, final_states


def gated_delta_bwd(q, k, v, dt, dt_bias, A, beta, dy, init_states=None, lengths=None,
                    scale: float = 1.0, dfinal_states=None, out_dtype=None, workspace=None, out=None):
    """Gradients of <dy, y> + <dfinal_states, final_states> of ``gated_delta_fwd``
    (``ssd_gated_delta_bwd``): a dict with dq, dk, dv, ddt and dbeta in ``out_dtype`` (v's
    type), and dA, ddt_bias and, with init_states, dinit_states in float32 (a given one must
    not overlap dfinal_states)."""
    lib = _native_lib()
    dev, shape, (B, T, H, P, N, G), odt, p = _delta_inputs(q, k, v, dt, dt_bias, A, beta, 4, scale,
                                                           out_dtype)
    ip = _check(init_states, "init_states", (B, H, P, N), _F32, dev)
    lp = _check(lengths, "lengths", (B,), _I32, dev)
    gp = _check(dy, "dy", (B, T, H, P), v.dtype, dev)
    fp = _check(dfinal_states, "dfinal_states", (B, H, P, N), _F32, dev)
    want = [("dq", (B, T, G, N), odt), ("dk", (B, T, G, N), odt), ("dv", (B, T, H, P), odt),
            ("ddt", (B, T, H), odt), ("dbeta", (B, T, H), odt), ("dA", (H,), _F32),
            ("ddt_bias", (H,), _F32)]
    if init_states is not None:
        want.append(("dinit_states", (B, H, P, N), _F32))
    out = _outputs(out, want, v)
    ws = _scratch(max(lib.ssd_gated_delta_bwd_workspace_size(shape), 1), v, workspace)
    st = lib.ssd_gated_delta_bwd(
        shape, *p, ip, lp, gp, fp, *(_at(out.get(n)) for n in (
            "dq", "dk", "dv", "ddt", "dbeta", "dA", "ddt_bias", "dinit_states")),
        ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_gated_delta_bwd", st)
    return out


def gated_delta_step(q, k, v, dt, dt_bias, A, beta, state, slots=None, scale: float = 1.0,
                     out_dtype=None, y=None):
    """One token of ``gated_delta_fwd`` (``ssd_gated_delta_step``): q, k (batch, ngroups,
    dstate), v, y (batch, nheads, headdim), dt, beta (batch, nheads); state (nslots, nheads,
    headdim, dstate) float32, updated in place; slots (batch,) int32 names each row's state, a
    negative one marks an empty row, whose output is 0.  dstate <= 256."""
    lib, vs, qs, ss, xd, dev = _native_lib(), v.shape, q.shape, state.shape, v.dtype, v.get_device()
    if (dev >= 0 and dev == _current_device() and len(vs) == 3 and len(qs) == 3 and xd in _CODE
            and out_dtype is None and y is None and v.is_contiguous()
            and qs[0] == vs[0] and q.dtype is xd and q.get_device() == dev and q.is_contiguous()
            and k.shape == qs and k.dtype is xd and k.get_device() == dev and k.is_contiguous()
            and dt.shape == vs[:2] and dt.dtype is xd and dt.get_device() == dev
            and dt.is_contiguous()
            and beta.shape == vs[:2] and beta.dtype is xd and beta.get_device() == dev
            and beta.is_contiguous()
            and ss == (ss[0], vs[1], vs[2], qs[2]) and state.dtype is _F32
            and state.get_device() == dev and state.is_contiguous()
            and A.shape == vs[1:2] and A.dtype is _F32 and A.get_device() == dev
            and A.is_contiguous()
            and (dt_bias is None or (dt_bias.shape == vs[1:2] and dt_bias.dtype is _F32
                                     and dt_bias.get_device() == dev and dt_bias.is_contiguous()))
            and (slots is None or (slots.shape == vs[:1] and slots.dtype is _I32
                                   and slots.get_device() == dev and slots.is_contiguous()))):
        code = _CODE[xd]
        shape = _native.DeltaShape(vs[0], 1, vs[1], vs[2], qs[2], qs[1], 0, 0, 0, 0, 0, 0, scale,
                                   code, code)
        y = _empty_like(v)
        st = lib.ssd_gated_delta_step(
            shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(),
            None if dt_bias is None else dt_bias.data_ptr(), A.data_ptr(), beta.data_ptr(),
            state.data_ptr(), None if slots is None else slots.data_ptr(), ss[0], y.data_ptr(),
            _stream(dev))
    else:
        dev, shape, (B, _, H, P, N, G), odt, p = _delta_inputs(q, k, v, dt, dt_bias, A, beta, 3,
                                                               scale, out_dtype)
        if state.dim() != 4:
            raise ValueError("state must be (nslots, nheads, headdim, dstate)")
        sp = _check(state, "state", (state.shape[0], H, P, N), _F32, dev)
        lp = _check(slots, "slots", (B,), _I32, dev)
        y = _output(y, "y", (B, H, P), odt, v)
        st = lib.ssd_gated_delta_step(shape, *p, sp, lp, state.shape[0], y.data_ptr(), _stream(dev))
    if st:
        _fail("ssd_gated_delta_step", st)
    return y


# ------------------------------------------------- norm of queries and keys

def _qk_inputs(q, k, w_q, w_k, freq, positions, l2, interleaved, eps, out_dtype):
    ndim = q.dim()
    if ndim not in (3, 4) or k.dim() != ndim:
        raise ValueError("q and k must be (batch, seqlen, heads, headdim), or (batch, heads, "
                         "headdim) for one token each")
    dev = _device(q)
    qshape, xd, lead = q.shape, q.dtype, ndim - 2
    HK, D = k.shape[-2], qshape[-1]
    qp, qs, qb = _rows(q, "q", qshape, lead, xd, dev)
    kp, ks, kb = _rows(k, "k", qshape[:lead] + (HK, D), lead, xd, dev)
    wq = None if w_q is None else _check(w_q, "w_q", (D,), _F32, dev)
    wk = None if w_k is None else _check(w_k, "w_k", (D,), _F32, dev)
    R, fp, pp = 0, None, None
    if freq is not None:
        if freq.dim() != 1 or 2 * freq.shape[0] > D:
            raise ValueError(f"freq: expected up to {D // 2} frequencies, got {tuple(freq.shape)}")
        R = 2 * freq.shape[0]
        fp = _check(freq, "freq", freq.shape, _F32, dev)
        if positions is None and ndim == 3 and R:
            raise ValueError("positions: required with freq where each row is one token")
    if positions is not None:
        pp = _check(positions, "positions", qshape[:lead], _I32, dev)
    code = _code(xd)
    if out_dtype is None:
        out_dtype, ocode = xd, code
    else:
        ocode = _code(out_dtype)
    shape = _native.QkNormShape(qshape[0], qshape[1] if ndim == 4 else 1, qshape[-2], HK, D, R, qs, ks,
                                qb, kb, eps, 1 if l2 else 0, 1 if interleaved else 0, code, ocode)
    return dev, shape, out_dtype, (qp, kp, wq, wk, fp, pp)


def qk_norm_fwd(q, k, w_q=None, w_k=None, freq=None, positions=None, l2: bool = False,
                interleaved: bool = False, eps: float = 1e-6, out_dtype=None, q_out=None, k_out=None):
    """q_out, k_out = queries and keys normalised head by head and turned by their positions
    (``ssd_qk_norm_fwd``): x / sqrt(mean(x^2) + eps) w (``l2``: x / sqrt(sum(x^2) + eps) w),
    then the pairs (i, i + n) of the first 2 n columns, n = len(freq), by the angles
    position * freq[i] (``interleaved``: the pairs (2 i, 2 i + 1)).

    q (batch, seqlen, q_heads, headdim), k (batch, seqlen, k_heads, headdim), or without
    seqlen for one token a row; both may be column ranges of wider tensors.  w_q, w_k
    (headdim,) float32 or None; freq float32, None: no rotation; positions (batch, seqlen), or
    (batch,), int32; None: 0, 1, ... along seqlen.  headdim <= 1024."""
    lib, qs, ks, xd, dev = _native_lib(), q.shape, k.shape, q.dtype, q.get_device()
    n, st, sk = len(qs), q.stride(), k.stride()
    # (a decoding step's call, as in layer_ops: its checks in one condition)
    if (n > 2 and dev >= 0 and dev == _current_device() and xd in _CODE and out_dtype is None
            and q_out is None and k_out is None and n < 5 and len(ks) == n
            and ks[:n - 2] == qs[:n - 2] and ks[n - 1] == qs[n - 1] and k.dtype is xd
            and k.get_device() == dev
            and st[n - 1] == 1 and sk[n - 1] == 1 and st[n - 2] == qs[n - 1] and sk[n - 2] == qs[n - 1]
            and st[n - 3] >= qs[n - 2] * qs[n - 1] and sk[n - 3] >= ks[n - 2] * qs[n - 1]
            and (w_q is None or (w_q.shape == qs[n - 1:] and w_q.dtype is _F32
                                 and w_q.get_device() == dev and w_q.is_contiguous()))
            and (w_k is None or (w_k.shape == qs[n - 1:] and w_k.dtype is _F32
                                 and w_k.get_device() == dev and w_k.is_contiguous()))
            and (positions is None or (positions.shape == qs[:n - 2] and positions.dtype is _I32
                                       and positions.get_device() == dev and positions.is_contiguous()))
            and (freq is None or (freq.dim() == 1 and freq.dtype is _F32 and freq.get_device() == dev
                                  and freq.is_contiguous() and 2 * freq.shape[0] <= qs[n - 1]
                                  and (n == 4 or positions is not None)))):
        code = _CODE[xd]
        shape = _native.QkNormShape(qs[0], qs[1] if n == 4 else 1, qs[n - 2], ks[n - 2], qs[n - 1],
                                    0 if freq is None else 2 * freq.shape[0], st[n - 3], sk[n - 3],
                                    st[0], sk[0], eps, 1 if l2 else 0, 1 if interleaved else 0, code, code)
        q_out = _empty(qs, dtype=xd, device=q.device)
        k_out = _empty(ks, dtype=xd, device=q.device)
        st = lib.ssd_qk_norm_fwd(
            shape, q.data_ptr(), k.data_ptr(), None if w_q is None else w_q.data_ptr(),
            None if w_k is None else w_k.data_ptr(), None if freq is None else freq.data_ptr(),
            None if positions is None else positions.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
            _stream(dev))
    else:
        dev, shape, odt, p = _qk_inputs(q, k, w_q, w_k, freq, positions, l2, interleaved, eps, out_dtype)
        q_out = _output(q_out, "q_out", q.shape, odt, q)
        k_out = _output(k_out, "k_out", k.shape, odt, q)
        st = lib.ssd_qk_norm_fwd(shape, *p, q_out.data_ptr(), k_out.data_ptr(), _stream(dev))
    if st:
        _fail("ssd_qk_norm_fwd", st)
    return q_out, k_out


def qk_norm_bwd(q, k, w_q, w_k, freq, positions, dq_out, dk_out, l2: bool = False,
                interleaved: bool = False, eps: float = 1e-6, out_dtype=None, workspace=None, out=None):
    """Gradients of <dq_out, q_out> + <dk_out, k_out> of ``qk_norm_fwd`` from its inputs
    (``ssd_qk_norm_bwd``): a dict with dq, dk (``out_dtype``, q's type) and, with w_q and w_k,
    dw_q and dw_k (float32), summed over tokens and heads."""
    lib = _native_lib()
    dev, shape, odt, p = _qk_inputs(q, k, w_q, w_k, freq, positions, l2, interleaved, eps, out_dtype)
    gq = _check(dq_out, "dq_out", q.shape, q.dtype, dev)
    gk = _check(dk_out, "dk_out", k.shape, q.dtype, dev)
    D = q.shape[-1:]
    want = [("dq", q.shape, odt), ("dk", k.shape, odt)]
    want += [(n, D, _F32) for n, w in (("dw_q", w_q), ("dw_k", w_k)) if w is not None]
    out = _outputs(out, want, q)
    ws = _scratch(max(lib.ssd_qk_norm_workspace_size(shape), 1), q, workspace)
    st = lib.ssd_qk_norm_bwd(shape, *p, gq, gk, out["dq"].data_ptr(), out["dk"].data_ptr(),
                             _at(out.get("dw_q")), _at(out.get("dw_k")), ws.data_ptr(),
                             ws.numel() * ws.element_size(), _stream(dev))
    if st:
        _fail("ssd_qk_norm_bwd", st)
    return out
