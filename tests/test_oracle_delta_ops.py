"""Pins of the fp64 oracle of the gated delta rule and of the norm of queries and keys
(CPU): closed forms, resuming from states, and gradients against central differences (step
1e-6: truncation ~1e-12, cancellation ~1e-10 of the loss, so 1e-6 of the largest gradient
has three digits to spare)."""
import numpy as np
import pytest

from oracle import delta_ops as do
from test_oracle_layer_ops import differences, rng


def inputs(seed, B=2, T=5, H=4, G=2, P=3, N=4):
    g = rng(seed)
    return dict(q=g.standard_normal((B, T, G, N)) * 0.6, k=g.standard_normal((B, T, G, N)) * 0.6,
                v=g.standard_normal((B, T, H, P)), dt=g.standard_normal((B, T, H)) - 1.0,
                dt_bias=g.standard_normal(H) * 0.3, A=-np.exp(g.standard_normal(H) * 0.3),
                beta=g.standard_normal((B, T, H)), init=g.standard_normal((B, H, P, N)))


@pytest.mark.parametrize("lengths", [None, [5, 0], [1, 4]])
def test_delta_gradients_are_differences(lengths):
    a = inputs(1)
    g = rng(2)
    dy, df = g.standard_normal((2, 5, 4, 3)), g.standard_normal((2, 4, 3, 4))

    def loss(q, k, v, dt, dt_bias, A, beta, init):
        y, fin = do.delta_fwd(q, k, v, dt, dt_bias, A, beta, init, lengths, 0.7)
        return float((y * dy).sum() + (fin * df).sum())
    r = do.delta_bwd(*list(a.values())[:7], dy, a["init"], lengths, 0.7, df)
    differences(loss, a, a, {n: r["d" + n] if n != "init" else r["dinit_states"] for n in a})


def test_delta_resumes_from_its_state():
    a = inputs(3, T=7)
    args = list(a.values())
    y, fin = do.delta_fwd(*args)
    cut = lambda s: [m[:, s] if m.ndim > 2 else m for m in args[:7]]  # noqa: E731
    y1, f1 = do.delta_fwd(*cut(slice(0, 3)), a["init"])
    y2, f2 = do.delta_fwd(*cut(slice(3, 7)), f1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-13) and np.allclose(f2, fin, atol=1e-13)


def test_delta_of_orthonormal_keys_is_a_table():
    """No decay, full strength, keys from an orthonormal set: a key's last value is
    what its query reads."""
    T, N = 6, 4
    g = rng(4)
    order = [0, 2, 1, 2, 0, 3]
    eye = np.linalg.qr(g.standard_normal((N, N)))[0]
    k = eye[order][None, :, None, :]
    v = g.standard_normal((1, T, 1, 2))
    big = np.full((1, T, 1), 60.0)
    y, S = do.delta_fwd(k, k, v, -big, None, np.zeros(1), big)
    assert np.allclose(y, v, atol=1e-12)
    for n, t in ((0, 4), (1, 2), (2, 3), (3, 5)):
        assert np.allclose(S[0, 0] @ eye[n], v[0, t, 0], atol=1e-12)


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [0, 2, 3])
def test_norm_gradients_are_differences(l2, interleaved, pairs):
    g = rng(pairs)
    a = dict(x=g.standard_normal((4, 2, 6)), w=1.0 + 0.1 * g.standard_normal(6))
    freq, pos = g.uniform(0.1, 1.0, pairs), np.array([0, 3, -2, 9])
    dy = g.standard_normal((4, 2, 6))

    def loss(x, w):
        return float((do.norm_fwd(x, w, freq, pos, l2, interleaved) * dy).sum())
    dx, dw = do.norm_bwd(a["x"], a["w"], freq, pos, dy, l2, interleaved)
    differences(loss, a, a, dict(x=dx, w=dw))


def test_rotation_keeps_lengths_and_differences_of_positions():
    g = rng(5)
    x, freq = g.standard_normal((1, 1, 8)), np.array([1.0, 0.3, 0.1, 0.03])
    y = np.concatenate([do.norm_fwd(x, None, freq, [p], eps=0.0) for p in (0, 5, 9, 14)])[:, 0]
    assert np.allclose((y * y).sum(-1), 8.0)
    assert np.isclose(y[0] @ y[1], y[2] @ y[3])
    z = do.norm_fwd(x, None, freq, [np.pi / 2], l2=True, interleaved=True, eps=0.0)[0, 0]
    u = x[0, 0] / np.linalg.norm(x)
    assert np.allclose(z[:2], [-u[1], u[0]])
