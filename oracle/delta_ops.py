"""The gated delta rule and the norm of queries and keys in fp64 numpy -- TEST
INFRASTRUCTURE (see ``oracle``).

Written from the formulas, one token at a time, sharing no code with the CUDA
library:

  gated delta rule   a = exp(softplus(dt + dt_bias) A),  b = sigmoid(beta)
                     S <- a S,  S <- S + b (v - S k) k^T,  y = scale S q
  norm               n = x / sqrt(mean(x^2) + eps) w   (l2: sum),  pairs (c, e) of n's first
                     columns turned:  c + i e  ->  (c + i e) exp(i position freq)

``lengths[b]``: positions from there on are padding (output and gradients 0, the state
stays).  Pins: ``tests/test_oracle_delta_ops.py``.
"""
from __future__ import annotations

import numpy as np

from .gated_norm import sigmoid
from .layer_ops import _f64, _lengths, softplus


# -------------------------------------------------------- gated delta rule

def _gates(dt, dt_bias, A, beta, live):
    z = dt if dt_bias is None else dt + dt_bias
    delta = softplus(z) * live[..., None]
    return z, delta, np.exp(delta * A), sigmoid(beta) * live[..., None]


def delta_fwd(q, k, v, dt, dt_bias, A, beta, init=None, lengths=None, scale=1.0, states=None):
    """(y (B, T, H, P), final (B, H, P, N)); appends the state in front of each token to
    the list ``states``."""
    q, k, v, dt, dt_bias, A, beta, init = _f64(q, k, v, dt, dt_bias, A, beta, init)
    B, T, H, P = v.shape
    rep = H // q.shape[2]
    live = (np.arange(T)[None] < _lengths(lengths, B, T)[:, None]).astype(float)
    _, _, a, b = _gates(dt, dt_bias, A, beta, live)
    S = np.zeros((B, H, P, q.shape[3])) if init is None else init.copy()
    y = np.zeros_like(v)
    for t in range(T):
        on = live[:, t].astype(bool)
        if states is not None:
            states.append(S.copy())
        kt = np.where(on[:, None, None], np.repeat(k[:, t], rep, 1), 0.0)
        qt = np.where(on[:, None, None], np.repeat(q[:, t], rep, 1), 0.0)
        vt = np.where(on[:, None, None], v[:, t], 0.0)
        S = a[:, t, :, None, None] * S
        u = b[:, t, :, None] * (vt - np.einsum("bhpn,bhn->bhp", S, kt))
        S = S + u[..., None] * kt[:, :, None, :]
        y[:, t] = scale * np.einsum("bhpn,bhn->bhp", S, qt)
    return y, S


def delta_bwd(q, k, v, dt, dt_bias, A, beta, dy, init=None, lengths=None, scale=1.0, dfinal=None):
    """dq, dk, dv, ddt, dbeta, dA, ddt_bias, dinit_states."""
    states = []
    delta_fwd(q, k, v, dt, dt_bias, A, beta, init, lengths, scale, states)
    q, k, v, dt, dt_bias, A, beta, dy, dfinal = _f64(q, k, v, dt, dt_bias, A, beta, dy, dfinal)
    B, T, H, P = v.shape
    G, N = q.shape[2:]
    rep = H // G
    live = (np.arange(T)[None] < _lengths(lengths, B, T)[:, None]).astype(float)
    z, delta, a, b = _gates(dt, dt_bias, A, beta, live)
    dS = np.zeros((B, H, P, N)) if dfinal is None else dfinal.copy()
    g = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), ddt=np.zeros_like(dt),
             dbeta=np.zeros_like(beta), dA=np.zeros_like(A))
    group = lambda m: m.reshape(B, G, rep, N).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        on = live[:, t].astype(bool)[:, None, None]
        kt, qt = (np.where(on, np.repeat(m[:, t], rep, 1), 0.0) for m in (k, q))
        vt, gy = np.where(on, v[:, t], 0.0), np.where(on, scale * dy[:, t], 0.0)
        bt = b[:, t, :, None]
        S0 = a[:, t, :, None, None] * states[t]
        e = vt - np.einsum("bhpn,bhn->bhp", S0, kt)
        S1 = S0 + (bt * e)[..., None] * kt[:, :, None, :]
        g["dq"][:, t] = group(np.einsum("bhpn,bhp->bhn", S1, gy))
        dS = dS + gy[..., None] * qt[:, :, None, :]
        du = np.einsum("bhpn,bhn->bhp", dS, kt)              # of u = b e
        de = bt * du
        dk = np.einsum("bhpn,bhp->bhn", dS, bt * e) - np.einsum("bhpn,bhp->bhn", S0, de)
        g["dk"][:, t] = group(dk)
        g["dv"][:, t] = de
        s = b[:, t]
        g["dbeta"][:, t] = (du * e).sum(-1) * s * (1.0 - s)
        dS0 = dS - de[..., None] * kt[:, :, None, :]
        dlog = (dS0 * S0).sum((-1, -2))                      # of delta A
        g["dA"] += (dlog * delta[:, t]).sum(0)
        g["ddt"][:, t] = dlog * A * sigmoid(z[:, t]) * live[:, t, None]
        dS = a[:, t, :, None, None] * dS0
    g["ddt_bias"] = g["ddt"].sum((0, 1))
    g["dinit_states"] = dS
    return g


# ---------------------------------------------- norm of queries and keys

def _turn(n, pairs, interleaved, angle, back=False):
    """The first 2 pairs columns of n turned by angle (rows, 1, pairs)."""
    c, e = (n[..., 0:2 * pairs:2], n[..., 1:2 * pairs:2]) if interleaved else \
        (n[..., :pairs], n[..., pairs:2 * pairs])
    z = (c + 1j * e) * np.exp((-1j if back else 1j) * angle)
    out = n.copy()
    if interleaved:
        out[..., 0:2 * pairs:2], out[..., 1:2 * pairs:2] = z.real, z.imag
    else:
        out[..., :pairs], out[..., pairs:2 * pairs] = z.real, z.imag
    return out


def norm_fwd(x, w=None, freq=None, positions=None, l2=False, interleaved=False, eps=1e-6):
    """x (rows, heads, headdim), positions (rows,)."""
    x, w, freq = _f64(x, w, freq)
    ss = (x * x).sum(-1, keepdims=True)
    n = x / np.sqrt((ss if l2 else ss / x.shape[-1]) + eps)
    n = n if w is None else n * w
    if freq is None or len(freq) == 0:
        return n
    return _turn(n, len(freq), interleaved, np.asarray(positions, np.float64)[:, None, None] * freq)


def norm_bwd(x, w, freq, positions, dy, l2=False, interleaved=False, eps=1e-6):
    """dx, dw."""
    x, w, freq, dy = _f64(x, w, freq, dy)
    D = x.shape[-1]
    if freq is not None and len(freq):
        dy = _turn(dy, len(freq), interleaved, np.asarray(positions, np.float64)[:, None, None] * freq, True)
    ss = (x * x).sum(-1, keepdims=True)
    r = 1.0 / np.sqrt((ss if l2 else ss / D) + eps)
    g = dy if w is None else dy * w
    dx = r * g - x * r ** 3 * (g * x).sum(-1, keepdims=True) * (1.0 if l2 else 1.0 / D)
    return dx, (dy * x * r).sum((0, 1))
