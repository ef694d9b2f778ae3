"""The gated delta rule at values where it can go wrong -- gates that are not numbers, decays
that are 0, outliers, infinities, states that live long -- against the fp64 oracle
(``oracle/delta_ops.py``) on a GPU.  Tolerances are those of ``test_delta_ops`` (1e-5 in relative
L2 for fp32 outputs) unless a test derives its own."""
import numpy as np
import pytest

from oracle import delta_ops as do
from test_delta_ops import close, delta_case, dev, on_gpu, small, stored, types

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["dt", "beta", "dt_bias", "A"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [150, 1300])  # whole, and cut into segments
def test_a_gate_that_is_nan_reaches_what_it_should(cuda_lib, name, dtype, T):
    """From its token on, the head's outputs, its final state and what its gradients are sums
    over are NaN, and no other head's bits change."""
    import torch
    it, _ = types(dtype)
    a, init, dy, df, _ = delta_case(2, T, 2, 2, 24, 40, dtype, True, None)
    gy, more = dev(dy, it), dict(init_states=dev(init))
    want = cuda_lib.gated_delta_fwd(*on_gpu(a, it), **more)
    back = cuda_lib.gated_delta_bwd(*on_gpu(a, it), gy, dfinal_states=dev(df), **more)
    at = 70 if name in ("dt", "beta") else 0
    rows = slice(0, 1) if name in ("dt", "beta") else slice(0, 2)  # batch rows that it reaches
    if name in ("dt", "beta"):
        a[name][0, at, 1] = np.nan
    else:
        a[name][1] = np.nan
    x = on_gpu(a, it)
    y, fin = cuda_lib.gated_delta_fwd(*x, **more)
    got = cuda_lib.gated_delta_bwd(*x, gy, dfinal_states=dev(df), **more)
    assert bool(y[rows, at:, 1].isnan().all()) and bool(fin[rows, 1].isnan().all())
    assert torch.equal(y[:, :, 0], want[0][:, :, 0]) and torch.equal(fin[:, 0], want[1][:, 0])
    assert torch.equal(y[rows, :at // 64 * 64, 1], want[0][rows, :at // 64 * 64, 1])
    assert bool(got["ddt"][rows, :, 1].isnan().all()) and bool(got["dinit_states"][rows, 1].isnan().all())
    for n in ("dA", "ddt_bias"):
        assert bool(got[n][1].isnan()) and torch.equal(got[n][0], back[n][0])
    for n in ("dv", "ddt", "dbeta"):
        assert torch.equal(got[n][:, :, 0], back[n][:, :, 0])
    assert torch.equal(got["dinit_states"][:, 0], back["dinit_states"][:, 0])
    one = {n: m[:, at] if m.ndim > 2 else m for n, m in a.items()}
    state = dev(init)
    y1 = cuda_lib.gated_delta_step(*on_gpu(one, it), state)  # the token by itself agrees
    assert bool(y1[rows, 1].isnan().all()) and bool(state[rows, 1].isnan().all())
    assert bool(y1[:, 0].isfinite().all()) and bool(state[:, 0].isfinite().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("step", [300.0, 3e4, np.inf])
def test_gates_of_decays_that_are_zero(cuda_lib, dtype, step):
    """Steps that forget everything next to ordinary ones: their gates' gradients are 0, and
    the parameters' sums, which multiply by the step, are those of the others."""
    import torch
    it, _ = types(dtype)
    a, init, dy, df, _ = delta_case(1, 192, 2, 2, 16, 32, dtype, True, None)
    a["A"] = stored(np.array([-0.7, -2.0]), torch.float32)  # 300 steps: 2^-300 and less
    hard = np.random.default_rng(1).random((1, 192, 2)) < 0.1
    a["dt"] = stored(np.where(hard, step, a["dt"]), it)
    got = cuda_lib.gated_delta_bwd(*on_gpu(a, it), dev(dy, it), init_states=dev(init), dfinal_states=dev(df))
    # (the oracle multiplies by the step: a finite one whose decay is 0 as well)
    ref = do.delta_bwd(*dict(a, dt=np.where(hard, 3e4, a["dt"])).values(), dy, init, dfinal=df)
    close("ddt", got["ddt"], ref["ddt"])
    terms = np.sqrt((ref["ddt"] ** 2).sum())
    for n in ("dA", "ddt_bias"):
        small(n, got[n], ref[n], terms)
    assert not got["ddt"].cpu()[torch.from_numpy(hard)].any()


def relative(got, ref):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    return np.linalg.norm(g - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["f32", "mixed", "bf16"])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6])
@pytest.mark.parametrize("N", [40, 128])
def test_a_token_next_to_a_larger_one(cuda_lib, dtype, size, N):
    """What a token's outputs (gradients) do not depend on takes nothing from them: later
    (earlier) tokens of its chunk that are 1e6 times larger.  Operands hold 2^-39 of their row's
    largest value, 3 size: 5e-6 of a value at most and, uniform, 1.6e-6 in the mean square,
    which the usual 1e-5 covers.  bf16 outputs add half a step in the 8th bit, 2^-8."""
    import torch
    it, ot = types(dtype)
    a, init, dy, df, _ = delta_case(1, 100, 2, 1, 24, N, dtype, True, None)
    a["v"][0, 50] = stored(a["v"][0, 50] * size, it)
    dy[0, 10] = stored(dy[0, 10] * size, it)
    x, more = on_gpu(a, it), dict(init_states=dev(init), out_dtype=ot)
    y, _ = cuda_lib.gated_delta_fwd(*x, **more)
    yr, _ = do.delta_fwd(*a.values(), init)
    tol = 1e-5 + (2.0 ** -8 if ot == torch.bfloat16 else 0.0)
    assert relative(y[:, :50], yr[:, :50]) <= tol
    got = cuda_lib.gated_delta_bwd(*x, dev(dy, it), dfinal_states=dev(df), **more)
    ref = do.delta_bwd(*a.values(), dy, init, dfinal=df)
    assert relative(got["dv"][:, 11:], ref["dv"][:, 11:]) <= tol


@pytest.mark.parametrize("size", [1e2, 1e4, 1e6])
def test_columns_of_a_state_next_to_larger_ones(cuda_lib, size):
    """Keys along the axes: each column of a state holds its own values, of sizes that differ,
    and keeps them for the queries that read it alone (bounds as above)."""
    import torch
    a, init, _, _, _ = delta_case(1, 200, 2, 1, 24, 32, "f32", True, None)
    at = np.random.default_rng(0).integers(0, 32, 200)
    a["k"][0, :, 0] = a["q"][0, :, 0] = np.eye(32)[at]
    scale = np.where(np.arange(32) < 3, size, 1.0)
    a["v"] = stored(a["v"] * scale[at][None, :, None, None], torch.float32)
    init = stored(init * scale, torch.float32)
    y, fin = cuda_lib.gated_delta_fwd(*on_gpu(a, None), init_states=dev(init))
    yr, fr = do.delta_fwd(*a.values(), init)
    for big in (True, False):
        t, c = (at < 3) == big, (np.arange(32) < 3) == big
        assert relative(y[:, t], yr[:, t]) <= 1e-5
        assert relative(fin[..., c], fr[..., c]) <= 1e-5


@pytest.mark.parametrize("name,where", [
    ("v", (0, 60, 1, 3)), ("v", (0, 100, 0, 0)), ("k", (0, 60, 0, 5)), ("q", (0, 60, 0, 5)),
    ("dy", (0, 20, 1, 3)), ("init", (0, 1, 3, 5)), ("dfinal", (0, 1, 3, 5))])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_infinity_leaves_nothing_wrong(cuda_lib, name, where, value, dtype):
    """Results that are finite are right, and what the definition makes infinite or NaN is not
    finite."""
    import torch
    it, _ = types(dtype)
    a, init, dy, df, _ = delta_case(1, 150, 2, 1, 16, 32, dtype, True, None)
    dict(a, dy=dy, init=init, dfinal=df)[name][where] = value
    x, more = on_gpu(a, it), dict(init_states=dev(init), out_dtype=torch.float32)
    y, fin = cuda_lib.gated_delta_fwd(*x, **more)
    got = cuda_lib.gated_delta_bwd(*x, dev(dy, it), dfinal_states=dev(df), **more)
    with np.errstate(all="ignore"):
        yr, fr = do.delta_fwd(*a.values(), init)
        ref = do.delta_bwd(*a.values(), dy, init, dfinal=df)
    for n, g, r in [("y", y, yr), ("final", fin, fr)] + [(n, got[n], ref[n]) for n in got]:
        g = g.double().cpu().numpy()
        both = np.isfinite(g) & np.isfinite(r)
        assert not (np.isfinite(g) & ~np.isfinite(r)).any(), n
        if both.any():  # (dA, ddt_bias: 5e-5 of their terms, as in test_delta_ops)
            tol = 5e-5 if n in ("dA", "ddt_bias") else 1e-5
            top = np.linalg.norm(r[both])
            if n in ("dA", "ddt_bias"):
                top = max(top, np.linalg.norm(ref["ddt"][np.isfinite(ref["ddt"])]))
            assert np.linalg.norm((g - r)[both]) <= tol * top, n


@pytest.mark.parametrize("dtype", ["f32", "mixed"])
@pytest.mark.parametrize("H", [2, 64])  # cut into segments, and one chain over all chunks
def test_states_that_live_long(cuda_lib, dtype, H):
    """Slow decays and small strengths: the state of the last token holds what 8192 tokens of one
    sign added, so a bias of an addition would count 128 chunks' times.  A rounded addition a
    chunk, 2^-24 each and independent, is sqrt(128) of them, 7e-7, beside the usual errors."""
    import torch
    it, _ = types(dtype)
    T, G, P, N = 8192, 1, 4, 32
    g = np.random.default_rng(H)
    n = g.standard_normal
    unit = lambda m: m / np.linalg.norm(m, axis=-1, keepdims=True)  # noqa: E731
    a = dict(q=stored(unit(np.abs(n((1, T, G, N)))), it), k=stored(unit(np.abs(n((1, T, G, N)))), it),
             v=stored(1 + 0.3 * n((1, T, H, P)), it), dt=stored(n((1, T, H)) - 9, it),
             dt_bias=stored(0.1 * n(H), torch.float32), A=stored(-0.1 * np.exp(0.1 * n(H)), torch.float32),
             beta=stored(n((1, T, H)) - 9, it))
    init = stored(3 + 0.1 * n((1, H, P, N)), torch.float32)
    dy = stored(np.abs(n((1, T, H, P))), it)
    x, more = on_gpu(a, it), dict(init_states=dev(init), out_dtype=torch.float32)
    y, fin = cuda_lib.gated_delta_fwd(*x, **more)
    yr, fr = do.delta_fwd(*a.values(), init)
    close("y", y, yr)
    close("final", fin, fr)
    got = cuda_lib.gated_delta_bwd(*x, dev(dy, it), **more)
    ref = do.delta_bwd(*a.values(), dy, init)
    for n in ("dq", "dk", "dv", "ddt", "dbeta", "dinit_states"):
        close(n, got[n], ref[n])
