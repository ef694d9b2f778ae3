"""The layer operators in fp64 numpy -- TEST INFRASTRUCTURE (see ``oracle``).

Written from the formulas, one position at a time, sharing no code with the
CUDA library:

  causal convolution   u_t = bias + sum_k w_k x_{t-K+1+k},  y = silu(u) or u
  selective scan       delta = softplus(dt + dt_bias)
                       h <- exp(delta A) h + delta x B,  y = C.h + D x,  out = y silu(z)
  block norm           t = o rstd(o) w_post,  r' = r + s gate t,  h = r' rstd(r') w_pre

``lengths[b]``: positions from there on are padding (output and gradients 0,
the state stays).  Pins: ``tests/test_oracle_layer_ops.py``.
"""
from __future__ import annotations

import numpy as np

from .gated_norm import sigmoid, silu, silu_grad


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def softplus(v):
    return np.logaddexp(0.0, v)


def _lengths(lengths, B, T):
    n = np.full(B, T) if lengths is None else np.asarray(lengths)
    return np.clip(n, 0, T).astype(int)


# ------------------------------------------------------------- convolution

def _padded(x, K, init):
    B, _, C = x.shape
    pre = np.zeros((B, K - 1, C)) if init is None else init
    return np.concatenate([pre, x], axis=1)


def conv_fwd(x, w, bias=None, init=None, lengths=None, silu_on=True):
    """(y (B, T, C), final (B, K - 1, C))."""
    x, w, bias, init = _f64(x, w, bias, init)
    B, T, C = x.shape
    K = w.shape[1]
    xp, n = _padded(x, K, init), _lengths(lengths, B, T)
    y = np.zeros((B, T, C))
    for b in range(B):
        for t in range(n[b]):
            u = (w.T * xp[b, t:t + K]).sum(0) + (0.0 if bias is None else bias)
            y[b, t] = silu(u) if silu_on else u
    final = np.stack([xp[b, n[b]:n[b] + K - 1] for b in range(B)])
    return y, final


def conv_bwd(x, w, bias, dy, init=None, lengths=None, silu_on=True, dfinal=None):
    """dx, dw, dbias, dinit."""
    x, w, bias, dy, init, dfinal = _f64(x, w, bias, dy, init, dfinal)
    B, T, C = x.shape
    K = w.shape[1]
    xp, n = _padded(x, K, init), _lengths(lengths, B, T)
    dxp, dw, db = np.zeros_like(xp), np.zeros_like(w), np.zeros(C)
    for b in range(B):
        for t in range(n[b]):
            u = (w.T * xp[b, t:t + K]).sum(0) + (0.0 if bias is None else bias)
            du = dy[b, t] * (silu_grad(u) if silu_on else 1.0)
            dxp[b, t:t + K] += w.T * du
            dw += (xp[b, t:t + K] * du).T
            db += du
        if dfinal is not None:
            dxp[b, n[b]:n[b] + K - 1] += dfinal[b]
    return dict(dx=dxp[:, K - 1:], dw=dw, dbias=db, dinit_state=dxp[:, :K - 1])


# ---------------------------------------------------------- selective scan

def _channels(m, D):
    """(..., G, N) -> (..., D, N)."""
    return np.repeat(m, D // m.shape[-2], axis=-2)


def scan_fwd(x, dt, dt_bias, A, B, C, D=None, z=None, init=None, lengths=None):
    """(out (B, T, D), final (B, D, N))."""
    x, dt, dt_bias, A, B, C, D, z, init = _f64(x, dt, dt_bias, A, B, C, D, z, init)
    Bt, T, Dc = x.shape
    n = _lengths(lengths, Bt, T)
    h = np.zeros((Bt,) + A.shape) if init is None else init.copy()
    out = np.zeros_like(x)
    for t in range(T):
        live = (t < n)[:, None]
        delta = softplus(dt[:, t] + (0.0 if dt_bias is None else dt_bias)) * live
        Bc, Cc = _channels(B[:, t], Dc), _channels(C[:, t], Dc)
        h = np.exp(delta[..., None] * A) * h + (delta * x[:, t])[..., None] * Bc
        y = (h * Cc).sum(-1) + (0.0 if D is None else D * x[:, t])
        out[:, t] = (y if z is None else y * silu(z[:, t])) * live
    return out, h


def scan_bwd(x, dt, dt_bias, A, B, C, D, z, dout, init=None, lengths=None, dfinal=None):
    x, dt, dt_bias, A, B, C, D, z, dout, init, dfinal = _f64(x, dt, dt_bias, A, B, C, D, z, dout,
                                                             init, dfinal)
    Bt, T, Dc = x.shape
    G, N = B.shape[2:]
    n = _lengths(lengths, Bt, T)
    hs = [np.zeros((Bt,) + A.shape) if init is None else init]
    deltas, ys = [], []
    for t in range(T):
        live = (t < n)[:, None]
        delta = softplus(dt[:, t] + (0.0 if dt_bias is None else dt_bias)) * live
        deltas.append(delta)
        hs.append(np.exp(delta[..., None] * A) * hs[-1]
                  + (delta * x[:, t])[..., None] * _channels(B[:, t], Dc))
        ys.append((hs[-1] * _channels(C[:, t], Dc)).sum(-1) + (0.0 if D is None else D * x[:, t]))
    g = np.zeros((Bt,) + A.shape) if dfinal is None else dfinal.copy()
    r = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dA=np.zeros_like(A), dB=np.zeros_like(B),
             dC=np.zeros_like(C), dD=np.zeros(Dc), ddt_bias=np.zeros(Dc), dz=np.zeros_like(x))
    for t in range(T - 1, -1, -1):
        live = (t < n)[:, None]
        dy = dout[:, t] * live
        if z is not None:
            r["dz"][:, t] = dy * ys[t] * silu_grad(z[:, t])
            dy = dy * silu(z[:, t])
        delta, Bc, Cc = deltas[t], _channels(B[:, t], Dc), _channels(C[:, t], Dc)
        g = g + dy[..., None] * Cc
        a = np.exp(delta[..., None] * A)
        gb = (g * Bc).sum(-1)
        w = g * a * hs[t]
        dv = ((w * A).sum(-1) + gb * x[:, t]) * live
        dv = dv * sigmoid(dt[:, t] + (0.0 if dt_bias is None else dt_bias))
        r["dx"][:, t] = gb * delta + (0.0 if D is None else D * dy)
        r["ddt"][:, t] = dv
        r["dA"] += (w * delta[..., None]).sum(0)
        r["dB"][:, t] = (g * (delta * x[:, t])[..., None]).reshape(Bt, G, Dc // G, N).sum(2)
        r["dC"][:, t] = (hs[t + 1] * dy[..., None]).reshape(Bt, G, Dc // G, N).sum(2)
        r["dD"] += (dy * x[:, t]).sum(0)
        r["ddt_bias"] += dv.sum(0)
        g = a * g
    r["dinit_states"] = g
    return r


# --------------------------------------------------------------- block norm

def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def block_norm_fwd(r, o, w_pre, w_post=None, gate=None, scale=1.0, eps=1e-5):
    """(r', h), rows x features."""
    r, o, w_pre, w_post, gate = _f64(r, o, w_pre, w_post, gate)
    t = o if w_post is None else o * _rstd(o, eps) * w_post
    if gate is not None:
        t = t * np.repeat(gate, r.shape[0] // gate.shape[0], axis=0)
    rn = r + scale * t
    return rn, rn * _rstd(rn, eps) * w_pre


def block_norm_bwd(r, o, w_pre, w_post, gate, dh, drout=None, scale=1.0, eps=1e-5):
    r, o, w_pre, w_post, gate, dh, drout = _f64(r, o, w_pre, w_post, gate, dh, drout)
    rows, F = r.shape
    ro = None if w_post is None else _rstd(o, eps)
    oh = o if w_post is None else o * ro
    t = oh if w_post is None else oh * w_post
    gt = None if gate is None else np.repeat(gate, rows // gate.shape[0], axis=0)
    rn = r + scale * (t if gate is None else gt * t)
    rr = _rstd(rn, eps)
    xh = rn * rr
    gx = dh * w_pre
    dr = rr * (gx - xh * (gx * xh).mean(-1, keepdims=True))
    if drout is not None:
        dr = dr + drout
    out = dict(dresidual=dr, dw_pre=(dh * xh).sum(0))
    dt = scale * dr
    if gate is not None:
        out["dgate"] = (dt * t).reshape(gate.shape[0], -1, F).sum(1)
        dt = dt * gt
    if w_post is not None:
        out["dw_post"] = (dt * oh).sum(0)
        gy = dt * w_post
        dt = ro * (gy - oh * (gy * oh).mean(-1, keepdims=True))
    out["do"] = dt
    return out


# -------------------------------------------------------------- SSD, one token

def ssd_step(x, dt, dt_bias, A, B, C, D, state):
    """(y (B, H, P), new state (B, H, P, N)) of one position of the SSD scan."""
    x, dt, dt_bias, A, B, C, D, state = _f64(x, dt, dt_bias, A, B, C, D, state)
    H = x.shape[1]
    delta = softplus(dt + (0.0 if dt_bias is None else dt_bias))
    Bh, Ch = _channels(B, H), _channels(C, H)
    h = np.exp(delta * A)[..., None, None] * state \
        + (delta[..., None] * x)[..., None] * Bh[:, :, None, :]
    y = (h * Ch[:, :, None, :]).sum(-1)
    if D is not None:
        y = y + D[:, None] * x
    return y, h
