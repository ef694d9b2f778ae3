"""Pins of the layer operators' fp64 oracle (CPU): closed forms, agreement with
the SSD oracle, resuming from states, and its gradients against central
differences (step 1e-6: truncation ~1e-12, cancellation ~1e-10 of the loss, so
1e-6 of the largest gradient has three digits to spare)."""
import numpy as np
import pytest

import oracle
from oracle import layer_ops as lo


def rng(seed):
    return np.random.default_rng(seed)


def differences(f, arrays, names, grads, seed=0):
    """Random directional differences of the scalar f against the gradients."""
    g = rng(seed)
    for k in names:
        for _ in range(3):
            v = g.standard_normal(arrays[k].shape)
            e = 1e-6
            up = f(**{**arrays, k: arrays[k] + e * v})
            dn = f(**{**arrays, k: arrays[k] - e * v})
            want = float((grads[k] * v).sum())
            assert abs((up - dn) / (2 * e) - want) <= 1e-6 * (1.0 + np.abs(grads[k]).sum()), k


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("silu_on", [True, False])
@pytest.mark.parametrize("lengths", [None, [5, 0, 1]])
def test_conv_gradients_are_differences(K, silu_on, lengths):
    g = rng(K)
    a = dict(x=g.standard_normal((3, 5, 4)), w=g.standard_normal((4, K)),
             bias=g.standard_normal(4), init=g.standard_normal((3, K - 1, 4)))
    dy, df = g.standard_normal((3, 5, 4)), g.standard_normal((3, K - 1, 4))

    def loss(x, w, bias, init):
        y, fin = lo.conv_fwd(x, w, bias, init, lengths, silu_on)
        return float((y * dy).sum() + (fin * df).sum())
    r = lo.conv_bwd(a["x"], a["w"], a["bias"], dy, a["init"], lengths, silu_on, df)
    differences(loss, a, a, dict(x=r["dx"], w=r["dw"], bias=r["dbias"], init=r["dinit_state"]))


def test_conv_identity_tap_and_resume():
    g = rng(1)
    x, w = g.standard_normal((2, 9, 3)), np.zeros((3, 4))
    w[:, 3] = 1.0
    y, fin = lo.conv_fwd(x, w, silu_on=False)
    assert np.array_equal(y, x) and np.array_equal(fin, x[:, -3:])
    w = g.standard_normal((3, 4))
    y, fin = lo.conv_fwd(x, w)
    y1, f1 = lo.conv_fwd(x[:, :2], w)
    y2, f2 = lo.conv_fwd(x[:, 2:], w, init=f1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-14) and np.array_equal(f2, fin)


def scan_inputs(seed, Bt=2, T=6, D=6, N=3, G=2):
    g = rng(seed)
    return dict(x=g.standard_normal((Bt, T, D)), dt=g.standard_normal((Bt, T, D)) - 1.0,
                dt_bias=g.standard_normal(D) * 0.3, A=-np.exp(g.standard_normal((D, N)) * 0.5),
                B=g.standard_normal((Bt, T, G, N)), C=g.standard_normal((Bt, T, G, N)),
                D=g.standard_normal(D), z=g.standard_normal((Bt, T, D)),
                init=g.standard_normal((Bt, D, N)))


@pytest.mark.parametrize("lengths", [None, [6, 2], [0, 1]])
@pytest.mark.parametrize("gated", [True, False])
def test_scan_gradients_are_differences(lengths, gated):
    a = scan_inputs(3)
    if not gated:
        a["z"] = None
    g = rng(4)
    dout, df = g.standard_normal(a["x"].shape), g.standard_normal(a["init"].shape)

    def loss(**kw):
        out, fin = lo.scan_fwd(lengths=lengths, **{**a, **kw})
        return float((out * dout).sum() + (fin * df).sum())
    r = lo.scan_bwd(a["x"], a["dt"], a["dt_bias"], a["A"], a["B"], a["C"], a["D"], a["z"], dout,
                    a["init"], lengths, df)
    names = dict(x="dx", dt="ddt", dt_bias="ddt_bias", A="dA", B="dB", C="dC", D="dD",
                 init="dinit_states")
    if gated:
        names["z"] = "dz"
    differences(loss, {k: a[k] for k in names}, names, {k: r[v] for k, v in names.items()})


def test_scan_equals_ssd_oracle_when_the_decay_is_the_heads():
    """P channels of a head with equal dt, A rows equal to the head's decay: the
    SSD recurrence."""
    Bt, T, H, P, N, G = 2, 7, 4, 3, 5, 2
    g = rng(6)
    x, dt = g.standard_normal((Bt, T, H, P)), g.standard_normal((Bt, T, H)) - 1.0
    bias, A, D = g.standard_normal(H), -np.exp(g.standard_normal(H)), g.standard_normal(H)
    B, C = g.standard_normal((Bt, T, G, N)), g.standard_normal((Bt, T, G, N))
    init = g.standard_normal((Bt, H, P, N))
    rep = lambda v: np.repeat(v, P, axis=-1)  # noqa: E731
    out, fin = lo.scan_fwd(x.reshape(Bt, T, H * P), rep(dt), rep(bias),
                           np.repeat(rep(A)[:, None], N, 1), B, C, rep(D),
                           init=init.reshape(Bt, H * P, N))
    y, f = oracle.ssd_fwd(x, dt, bias, A, B, C, D, init)
    assert np.allclose(out.reshape(x.shape), y, atol=1e-12)
    assert np.allclose(fin.reshape(f.shape), f, atol=1e-12)
    # and one token of it, from the state before the last position
    _, before = oracle.ssd_fwd(x[:, :-1], dt[:, :-1], bias, A, B[:, :-1], C[:, :-1], D, init)
    ys, fs = lo.ssd_step(x[:, -1], dt[:, -1], bias, A, B[:, -1], C[:, -1], D, before)
    assert np.allclose(ys, y[:, -1], atol=1e-12) and np.allclose(fs, f, atol=1e-12)


def test_scan_padding_keeps_the_state():
    a = scan_inputs(8)
    out, fin = lo.scan_fwd(lengths=[4, 0], **a)
    cut = {k: (v[:, :4] if v.ndim > 1 and v.shape[1] == 6 and k not in ("A", "init") else v)
           for k, v in a.items()}
    out4, fin4 = lo.scan_fwd(**cut)
    assert np.allclose(out[0, :4], out4[0]) and np.all(out[0, 4:] == 0) and np.all(out[1] == 0)
    assert np.allclose(fin[0], fin4[0]) and np.array_equal(fin[1], a["init"][1])


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gates", [0, 1, 2, 6])
def test_block_norm_gradients_are_differences(post, gates):
    g = rng(gates)
    a = dict(r=g.standard_normal((6, 5)), o=g.standard_normal((6, 5)), w_pre=g.standard_normal(5))
    names = dict(r="dresidual", o="do", w_pre="dw_pre")
    if post:
        a["w_post"], names["w_post"] = g.standard_normal(5), "dw_post"
    if gates:
        a["gate"], names["gate"] = g.standard_normal((gates, 5)), "dgate"
    dh, dr = g.standard_normal((6, 5)), g.standard_normal((6, 5))

    def loss(**kw):
        rn, h = lo.block_norm_fwd(scale=0.7, **kw)
        return float((h * dh).sum() + (rn * dr).sum())
    r = lo.block_norm_bwd(a["r"], a["o"], a["w_pre"], a.get("w_post"), a.get("gate"), dh, dr, 0.7)
    differences(loss, a, names, {k: r[v] for k, v in names.items()})


def test_block_norm_of_a_constant_row():
    r, o = np.zeros((1, 4)), np.full((1, 4), 3.0)
    rn, h = lo.block_norm_fwd(r, o, np.ones(4), np.full(4, 2.0), eps=0.0, scale=0.5)
    assert np.allclose(rn, 1.0) and np.allclose(h, 1.0)  # 0.5 * (3 / 3) * 2, normed
