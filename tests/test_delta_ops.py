"""The gated delta rule and the norm of queries and keys against the fp64 oracle
(``oracle/delta_ops.py``) on a GPU.

Tolerances.  Inputs are rounded to their storage type first, so the oracle sees the
kernels' values and what is left is the kernels' own arithmetic.  Products take operands
good to 2^-23 of a row's largest value (two planes of fp16, or three of bf16 at 2^-25), and
add up in fp32 by an instruction that truncates: up to 48 additions of one sign at half an
ulp, 48 x 3e-8 = 1.4e-6 of an element, through about four products one after another.  With
their roundings mostly independent that is under 1e-5 in relative L2, and 4e-5 of the
largest value anywhere.  A bf16 output has one more rounding, half a unit in the 8th bit:
2^-8 of the value, and where it alone depends on a product its operands are two planes of
bf16, 2^-16.  The gradients of A and dt_bias are sums over tokens of running sums in which
up to 64 terms of either sign cancel: sqrt(64) x 2e-6 of the terms' size, which is up to
three times the sums', so 5e-5."""
import numpy as np
import pytest

from oracle import delta_ops as do
from test_layer_ops import close, dev, stored, types

pytestmark = pytest.mark.gpu


def delta_case(B, T, H, G, P, N, dtype, has_init, lengths, seed=0, unit=True, dt_shift=-3.0):
    """Inputs as numpy, rounded to their type: unit keys and queries, steps around e^-3."""
    import torch
    it, _ = types(dtype)
    g = np.random.default_rng(seed + 1000 * B + T + 7 * P + N)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    q, k = n(B, T, G, N), n(B, T, G, N)
    if unit:
        q, k = (m / np.linalg.norm(m, axis=-1, keepdims=True) for m in (q, k))
    a = dict(q=stored(q, it), k=stored(k, it), v=stored(n(B, T, H, P), it),
             dt=stored(n(B, T, H) + dt_shift, it), dt_bias=stored(0.3 * n(H), torch.float32),
             A=stored(-np.exp(0.5 * n(H)), torch.float32), beta=stored(n(B, T, H), it))
    init = stored(0.5 * n(B, H, P, N), torch.float32) if has_init else None
    dy, df = stored(n(B, T, H, P), it), stored(0.3 * n(B, H, P, N), torch.float32)
    ln = np.array(lengths) if lengths is not None else None
    return a, init, dy, df, ln


def on_gpu(a, it):
    import torch
    return [dev(m, torch.float32 if name in ("A", "dt_bias") else it) for name, m in a.items()]


def small(name, got, ref, terms=1.0):
    """A gate's summed gradient; ``terms``: what it is a sum of, in size."""
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), name
    assert np.linalg.norm(g - ref) <= 5e-5 * max(np.linalg.norm(ref), terms) + 1e-30, name


DELTA = [
    # B, T, H, G, P, N, dtype, init, lengths
    (1, 1, 1, 1, 1, 1, "f32", False, None),
    (1, 1, 2, 1, 8, 16, "bf16", True, None),
    (2, 64, 2, 2, 16, 64, "f32", False, None),
    (2, 65, 4, 2, 40, 24, "f32", True, [65, 1]),
    (3, 130, 2, 1, 72, 100, "bf16", True, [130, 0, 64]),     # an empty row, a whole chunk
    (1, 200, 3, 3, 64, 128, "mixed", False, None),
    (2, 190, 6, 3, 128, 128, "bf16", True, None),
    (1, 129, 2, 1, 200, 128, "bf16", False, None),           # four tiles of value rows, a ragged one
    (1, 70, 8, 1, 24, 33, "bf16", True, None),               # rows that fill no 16 bytes
    (2, 100, 3, 1, 7, 65, "f32", True, [99, 100]),
    (1, 127, 5, 5, 33, 97, "mixed", True, None),
    (5, 63, 2, 2, 64, 64, "bf16", False, [0, 63, 5, 1, 62]),
]


@pytest.mark.parametrize("case", DELTA)
def test_delta_matches_oracle(cuda_lib, case):
    it, ot = types(case[6])
    a, init, dy, df, ln = delta_case(*case)
    x = on_gpu(a, it)
    import torch
    more = dict(init_states=dev(init), lengths=dev(ln, torch.int32), scale=0.5, out_dtype=ot)
    y, fin = cuda_lib.gated_delta_fwd(*x, **more)
    yr, fr = do.delta_fwd(*a.values(), init, ln, 0.5)
    close("y", y, yr)
    close("final", fin, fr)
    got = cuda_lib.gated_delta_bwd(*x, dev(dy, it), dfinal_states=dev(df), **more)
    ref = do.delta_bwd(*a.values(), dy, init, ln, 0.5, df)
    for n in ("dq", "dk", "dv", "ddt", "dbeta") + (("dinit_states",) if init is not None else ()):
        close(n, got[n], ref[n])
    terms = np.sqrt((ref["ddt"] ** 2).sum())
    for n in ("dA", "ddt_bias"):
        small(n, got[n], ref[n], terms)
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("case", [
    # few heads over many chunks: sequences long enough to be cut into segments, one that
    # ends inside one, one of them empty
    (3, 2100, 2, 1, 24, 40, "f32", True, [2100, 700, 0]),
    (2, 1500, 1, 1, 72, 128, "bf16", False, [1025, 1500]),
    (1, 4200, 2, 2, 16, 64, "mixed", True, None)])
def test_delta_of_long_sequences_of_few_heads(cuda_lib, case):
    test_delta_matches_oracle(cuda_lib, case)


def test_delta_without_bias_or_final_gradient(cuda_lib):
    a, _, dy, _, _ = delta_case(2, 77, 2, 1, 16, 16, "f32", False, None)
    x = [None if n == "dt_bias" else dev(m) for n, m in a.items()]
    a["dt_bias"] = None
    y, none = cuda_lib.gated_delta_fwd(*x, return_final_states=False)
    assert none is None
    close("y", y, do.delta_fwd(*a.values())[0])
    got, ref = cuda_lib.gated_delta_bwd(*x, dev(dy)), do.delta_bwd(*a.values(), dy)
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        close(n, got[n], ref[n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_of_repeated_keys(cuda_lib, dtype):
    """Every token has the same key: the chunk's system is full below its diagonal.  What a
    token writes replaces what the last one wrote, and the corrections of 64 tokens add up
    in each element: sqrt(64) times the usual 1e-5 / 4e-5."""
    import torch
    it, ot = types(dtype)
    a, init, dy, df, _ = delta_case(2, 150, 2, 1, 24, 40, dtype, True, None)
    a["k"][:] = a["k"][:, :1]
    x = on_gpu(a, it)
    y, fin = cuda_lib.gated_delta_fwd(*x, init_states=dev(init), out_dtype=torch.float32)
    yr, fr = do.delta_fwd(*a.values(), init)
    for n, got, ref in (("y", y, yr), ("final", fin, fr)):
        g = got.double().cpu().numpy()
        assert np.linalg.norm(g - ref) <= 8e-5 * np.linalg.norm(ref), n
    got = cuda_lib.gated_delta_bwd(*x, dev(dy, it), init_states=dev(init), out_dtype=torch.float32)
    ref = do.delta_bwd(*a.values(), dy, init)
    for n in ("dq", "dk", "dv", "dbeta", "dinit_states"):
        g = got[n].double().cpu().numpy()
        assert np.linalg.norm(g - ref[n]) <= 8e-5 * np.linalg.norm(ref[n]), n


@pytest.mark.parametrize("size", [1e-25, 1e-6, 1e4, 1e20])
def test_delta_of_values_of_any_size(cuda_lib, size):
    """y and the states are linear in the values and the initial state, so their size is
    nothing to the error relative to it (the fp16 planes' rows are scaled)."""
    a, init, _, _, _ = delta_case(1, 130, 2, 2, 32, 64, "f32", True, None)
    y0, f0 = do.delta_fwd(*a.values(), init)
    x = on_gpu(dict(a, v=a["v"] * size), None)
    y, fin = cuda_lib.gated_delta_fwd(*x, init_states=dev(init * size))
    close("y", y / size, y0)
    close("final", fin / size, f0)


def test_delta_of_keys_of_any_size(cuda_lib):
    """Keys of 1e-3 .. 30 in one chunk, with the strength such that b |k|^2 stays under 1."""
    import torch
    a, init, dy, df, _ = delta_case(1, 100, 2, 1, 16, 32, "f32", True, None)
    size = np.exp(np.random.default_rng(3).uniform(np.log(1e-3), np.log(30.0), (1, 100, 1)))
    a["k"] = stored(a["k"] * size[..., None], torch.float32)
    a["beta"] = stored(np.log(0.5 / np.maximum(size, 0.71) ** 2) + np.zeros_like(a["beta"]),
                       torch.float32)
    y, fin = cuda_lib.gated_delta_fwd(*on_gpu(a, None), init_states=dev(init))
    yr, fr = do.delta_fwd(*a.values(), init)
    for n, got, ref in (("y", y, yr), ("final", fin, fr)):
        g = got.double().cpu().numpy()
        assert np.linalg.norm(g - ref) <= 1e-5 * np.linalg.norm(ref), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_of_strong_decays_and_gates(cuda_lib, dtype):
    """Steps that forget everything next to steps that keep it, and strengths of 0 and 1."""
    it, _ = types(dtype)
    a, init, dy, df, _ = delta_case(1, 192, 2, 2, 16, 32, dtype, True, None)
    g = np.random.default_rng(1)
    hard = g.random((1, 192, 2)) < 0.1
    a["dt"] = stored(np.where(hard, 300.0, a["dt"]), it)
    a["beta"] = stored(np.where(g.random((1, 192, 2)) < 0.2, 60.0, np.where(hard, -200.0, a["beta"])), it)
    x = on_gpu(a, it)
    y, fin = cuda_lib.gated_delta_fwd(*x, init_states=dev(init))
    yr, fr = do.delta_fwd(*a.values(), init)
    close("y", y, yr)
    close("final", fin, fr)
    got = cuda_lib.gated_delta_bwd(*x, dev(dy, it), init_states=dev(init), dfinal_states=dev(df))
    ref = do.delta_bwd(*a.values(), dy, init, dfinal=df)
    for n in ("dq", "dk", "dv", "dbeta", "dinit_states"):
        close(n, got[n], ref[n])
    for n in ("ddt", "dA", "ddt_bias"):  # of decays that are 0 in fp32: 0
        assert bool(got[n].isfinite().all()), n


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [32, 33])
def test_delta_padding_reaches_nothing(cuda_lib, value, dtype, N):
    import torch
    it, _ = types(dtype)
    lengths = [70, 0, 128]
    a, init, dy, df, ln = delta_case(3, 130, 2, 1, 16, N, dtype, True, lengths)
    x, gy = on_gpu(a, it), dev(dy, it)
    more = dict(init_states=dev(init), lengths=dev(ln, torch.int32))
    want = cuda_lib.gated_delta_fwd(*x, **more)
    back = cuda_lib.gated_delta_bwd(*x, gy, dfinal_states=dev(df), **more)
    for m in [x[i] for i in (0, 1, 2, 3, 6)] + [gy]:
        for b, n in enumerate(lengths):
            m[b, n:] = value
    got = cuda_lib.gated_delta_fwd(*x, **more)
    again = cuda_lib.gated_delta_bwd(*x, gy, dfinal_states=dev(df), **more)
    for p, q in list(zip(want, got)) + [(back[k], again[k]) for k in back]:
        assert torch.equal(p, q)
    for b, n in enumerate(lengths):
        assert not got[0][b, n:].any() and not again["dq"][b, n:].any() and not again["ddt"][b, n:].any()
    assert torch.equal(got[1][1], more["init_states"][1])
    assert torch.equal(again["dinit_states"][1], dev(df)[1])


@pytest.mark.parametrize("dtype,shift", [("bf16", 0), ("bf16", 1), ("bf16", 8), ("f32", 0), ("f32", 3)])
def test_delta_of_column_ranges(cuda_lib, dtype, shift):
    """q, k and v as column ranges of one wider tensor, aligned and not."""
    import torch
    it, _ = types(dtype)
    a, init, dy, _, _ = delta_case(2, 100, 4, 2, 24, 32, dtype, False, None)
    x = on_gpu(a, it)
    wide = torch.full((2, 100, shift + 2 * 64 + 96 + 16), float("nan"), dtype=it, device="cuda")
    cut, at = [], shift
    for m in x[:3]:
        n = m.shape[2] * m.shape[3]
        wide[..., at:at + n] = m.flatten(2)
        cut.append(wide[..., at:at + n].unflatten(-1, m.shape[2:]))
        at += n
    want, got = cuda_lib.gated_delta_fwd(*x), cuda_lib.gated_delta_fwd(*cut, *x[3:])
    back = cuda_lib.gated_delta_bwd(*x, dev(dy, it))
    again = cuda_lib.gated_delta_bwd(*cut, *x[3:], dev(dy, it))
    for p, q in list(zip(want, got)) + [(back[k], again[k]) for k in back]:
        assert torch.equal(p, q)


def test_delta_past_32_bits(cuda_lib):
    """Batch rows further apart than 2^31 elements."""
    import torch
    a, _, dy, _, _ = delta_case(2, 80, 2, 1, 16, 32, "bf16", False, None)
    x = on_gpu(a, torch.bfloat16)
    apart = (1 << 31) + 64
    big = torch.empty(apart + 80 * 64, dtype=torch.bfloat16, device="cuda")
    far = []
    for m in x[:3]:
        n = m.shape[2] * m.shape[3]
        v = big.as_strided((2, 80) + tuple(m.shape[2:]), (apart, n, m.shape[3], 1), storage_offset=0)
        v.copy_(m)
        want = cuda_lib.gated_delta_fwd(*x)
        far = list(x)
        far[[t is m for t in x].index(True)] = v
        got = cuda_lib.gated_delta_fwd(*far)
        back, again = cuda_lib.gated_delta_bwd(*x, dev(dy, torch.bfloat16)), cuda_lib.gated_delta_bwd(
            *far, dev(dy, torch.bfloat16))
        for p, q in list(zip(want, got)) + [(back[k], again[k]) for k in back]:
            assert torch.equal(p, q)


def test_delta_gradients_are_differences(cuda_lib):
    """Along random directions of each input, in fp32.  The loss is a sum of ~10^4 terms of
    size 1, good to 1e-5 of their root sum 1e2: 1e-3; over a step that changes it by 10 each
    way that is 1e-4 of the difference, the curvature's share is of the same order, and 1 %
    leaves a factor of 50."""
    import torch
    a, init, dy, df, _ = delta_case(2, 97, 4, 2, 24, 32, "f32", True, None)
    x, s0 = on_gpu(a, None), dev(init)
    gy, gf = dev(dy), dev(df)

    def loss(args, s):
        y, fin = cuda_lib.gated_delta_fwd(*args, init_states=s, scale=0.7)
        return float((y.double() * gy).sum() + (fin.double() * gf).sum())
    got = cuda_lib.gated_delta_bwd(*x, gy, init_states=s0, scale=0.7, dfinal_states=gf)
    names = ("dq", "dk", "dv", "ddt", "ddt_bias", "dA", "dbeta")
    for i, n in enumerate(names + ("dinit_states",)):
        grad = got[n].double()
        v = grad / grad.norm()
        e = min(0.02 * float((x[i] if i < 7 else s0).norm()), 10.0 / float(grad.norm()))
        args = [list(x), list(x)]
        s = [s0, s0]
        for j, sign in enumerate((1.0, -1.0)):
            if i < 7:
                args[j][i] = (x[i].double() + sign * e * v).float()
            else:
                s[j] = (s0.double() + sign * e * v).float()
        diff = (loss(args[0], s[0]) - loss(args[1], s[1])) / (2 * e)
        assert abs(diff - float(grad.norm())) <= 1e-2 * float(grad.norm()), n


def test_repeats_are_bit_identical(cuda_lib):
    """Calls one after another, on another stream, and captured in a graph that is replayed
    with other work between: the same bits."""
    import torch
    a, init, dy, df, ln = delta_case(2, 150, 8, 2, 40, 100, "bf16", True, [150, 77])
    x, gy = on_gpu(a, torch.bfloat16), dev(dy, torch.bfloat16)
    more = dict(init_states=dev(init), lengths=dev(ln, torch.int32))
    q, k = x[0], x[1]
    freq = torch.linspace(1.0, 0.1, 25, device="cuda")
    w = torch.linspace(0.5, 1.5, 100, device="cuda")

    def everything():
        y, fin = cuda_lib.gated_delta_fwd(*x, **more)
        g = cuda_lib.gated_delta_bwd(*x, gy, dfinal_states=dev_df, **more)
        qo, ko = cuda_lib.qk_norm_fwd(q, k, w, w, freq)
        h = cuda_lib.qk_norm_bwd(q, k, w, w, freq, None, qo, ko)
        return [y, fin, *g.values(), qo, ko, *h.values()]
    dev_df = dev(df)
    first = [m.clone() for m in everything()]
    for _ in range(3):
        assert all(torch.equal(p, r) for p, r in zip(first, everything()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = everything()
    s.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(first, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = everything()
    for _ in range(2):
        for m in kept:
            m.fill_(7.0)
        g.replay()
        everything()
        assert all(torch.equal(p, r) for p, r in zip(first, kept))


# ---------------------------------------------------------------- one token

@pytest.mark.parametrize("B,H,G,P,N,dtype", [
    (1, 1, 1, 1, 1, "f32"), (3, 4, 2, 8, 16, "bf16"), (2, 6, 3, 40, 33, "f32"), (5, 2, 1, 64, 128, "mixed"),
    (2, 3, 1, 100, 100, "bf16"), (2, 2, 2, 7, 256, "bf16"), (1, 2, 2, 16, 130, "f32"), (2, 2, 1, 24, 255, "bf16"),
    (70, 8, 4, 64, 64, "bf16"), (64, 24, 12, 64, 128, "bf16"), (300, 4, 4, 64, 32, "f32")])
def test_delta_step_matches_oracle(cuda_lib, B, H, G, P, N, dtype):
    import torch
    it, ot = types(dtype)
    a, init, _, _, _ = delta_case(B, 1, H, G, P, N, dtype, True, None)
    one = {n: m[:, 0] if m.ndim > 2 else m for n, m in a.items()}
    state = dev(init)
    y = cuda_lib.gated_delta_step(*on_gpu(one, it), state, scale=0.5, out_dtype=ot)
    yr, fr = do.delta_fwd(*a.values(), init, None, 0.5)
    close("y", y, yr[:, 0])
    close("state", state, fr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_go_on_from_prompts(cuda_lib, dtype):
    """Ragged prompts by the chunked form, then tokens one by one on a cache of slots with
    an empty row, against one pass of the oracle over each whole sequence."""
    import torch
    it, _ = types(dtype)
    lengths, new = [70, 0, 64, 9], 5
    a, init, _, _, ln = delta_case(4, 75, 4, 2, 24, 32, dtype, True, lengths)
    x = on_gpu(a, it)
    prompt = [m[:, :70].contiguous() if m.dim() > 2 else m for m in x]
    _, fin = cuda_lib.gated_delta_fwd(*prompt, init_states=dev(init), lengths=dev(ln, torch.int32))
    slots = torch.tensor([5, 0, 3, 1, -1], dtype=torch.int32, device="cuda")
    cache = torch.full((7, 4, 24, 32), float("nan"), device="cuda")
    cache[slots[:4].long()] = fin
    untouched = cache[[2, 4, 6]].clone()
    yr, fr = do.delta_fwd(*a.values(), init, np.array(lengths) + new)
    for i in range(new):
        rows = [(b, n + i) for b, n in enumerate(lengths)] + [(0, 0)]
        tok = [torch.stack([m[b, n] for b, n in rows]) if m.dim() > 2 else m for m in x]
        y = cuda_lib.gated_delta_step(*tok, cache, slots=slots)
        close("y", y[:4], np.stack([yr[b, n] for b, n in rows[:4]]))
        assert not y[4].any()
    close("states", cache[slots[:4].long()], fr)
    assert torch.equal(cache[[2, 4, 6]].isnan(), untouched.isnan())


def test_step_empty_rows_and_column_ranges(cuda_lib):
    import torch
    a, init, _, _, _ = delta_case(4, 1, 4, 2, 24, 32, "bf16", True, None)
    one = on_gpu({n: m[:, 0] if m.ndim > 2 else m for n, m in a.items()}, torch.bfloat16)
    state = dev(init)
    want = cuda_lib.gated_delta_step(*one, state)
    for shift in (0, 1, 8):
        wide = torch.zeros(4, shift + 2 * 64 + 96, dtype=torch.bfloat16, device="cuda")
        cut, at = [], shift
        for m in one[:3]:
            n = m.shape[1] * m.shape[2]
            wide[:, at:at + n] = m.flatten(1)
            cut.append(wide[:, at:at + n].unflatten(-1, m.shape[1:]))
            at += n
        s2 = dev(init)
        assert torch.equal(cuda_lib.gated_delta_step(*cut, *one[3:], s2), want) and torch.equal(s2, state)
    slots = torch.tensor([-1, 1, 4, 2], dtype=torch.int32, device="cuda")  # 4: past the last slot
    for m in one[:4] + one[6:]:
        if m.dim() > 1:
            m[0] = float("nan")
            m[2] = float("inf")
    s3 = dev(init)
    y = cuda_lib.gated_delta_step(*one, s3, slots=slots)
    assert not y[0].any() and not y[2].any() and bool(y.isfinite().all())
    assert torch.equal(s3[[0, 3]], dev(init)[[0, 3]]) and not torch.equal(s3[1], dev(init)[1])


def test_step_of_a_cache_past_32_bits(cuda_lib):
    """A state cache of more than 2^31 elements: the last slot's state moves, and no other."""
    import torch
    slots_n = (1 << 31) // (4 * 64 * 128) + 3
    cache = torch.zeros(slots_n, 4, 64, 128, device="cuda")
    a, init, _, _, _ = delta_case(2, 1, 4, 2, 64, 128, "bf16", True, None)
    one = on_gpu({n: m[:, 0] if m.ndim > 2 else m for n, m in a.items()}, torch.bfloat16)
    at = torch.tensor([slots_n - 1, 1], dtype=torch.int32, device="cuda")
    cache[at.long()] = dev(init)
    small_cache = dev(init)
    want = cuda_lib.gated_delta_step(*one, small_cache)
    got = cuda_lib.gated_delta_step(*one, cache, slots=at)
    assert torch.equal(got, want) and torch.equal(cache[at.long()], small_cache)
    assert not cache[0].any() and not cache[2].any() and not cache[slots_n - 2].any()


# ------------------------------------------------- norm of queries and keys

def qk_case(lead, HQ, HK, D, R, dtype, weights, seed=0):
    import torch
    it, ot = types(dtype)
    g = np.random.default_rng(seed + D + R + 31 * HQ)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    a = dict(q=stored(n(*lead, HQ, D), it), k=stored(n(*lead, HK, D), it))
    w = [stored(1.0 + 0.2 * n(D), torch.float32) if weights else None for _ in range(2)]
    freq = stored(1e4 ** (-np.arange(R // 2) / max(1, R // 2)), torch.float32) if R else None
    gy = [stored(n(*lead, HQ, D), it), stored(n(*lead, HK, D), it)]
    return a, w, freq, gy, it, ot


QK = [
    # (batch, seqlen), q heads, k heads, D, rotary, dtype, weights, l2, interleaved, first position
    ((1, 1), 1, 1, 1, 0, "f32", True, False, False, 0),
    ((2, 5), 3, 1, 2, 2, "f32", True, False, True, 0),
    ((2, 9), 4, 2, 64, 64, "bf16", True, False, False, 0),
    ((1, 33), 5, 3, 128, 128, "bf16", True, False, True, 1000),
    ((2, 17), 8, 8, 128, 64, "mixed", False, True, False, 0),
    ((3, 7), 2, 5, 74, 38, "f32", True, False, True, 1 << 20),
    ((1, 20), 3, 2, 80, 32, "bf16", True, True, False, -50),
    ((1, 11), 2, 1, 256, 128, "f32", False, False, False, (1 << 31) - 20),
    ((2, 3), 1, 2, 1024, 512, "bf16", True, False, True, 7),
    ((1, 4), 1, 1, 1023, 1022, "f32", True, False, False, 3),
    ((1, 6), 2, 2, 24, 22, "bf16", True, False, False, -(1 << 31)),
    ((1, 5), 1, 1, 600, 600, "f32", True, True, False, 0),
    ((4, 600), 2, 1, 32, 32, "bf16", True, False, False, 0),
]


@pytest.mark.parametrize("case", QK)
def test_qk_norm_matches_oracle(cuda_lib, case):
    """Angles: the fp32 angle of a turn's fraction is off by 2^-25 of a half turn and its
    sine and cosine by 1e-7, as the other roundings here."""
    import torch
    (B, T), HQ, HK, D, R, dtype, weights, l2, inter, first = case
    a, w, freq, gy, it, ot = qk_case((B, T), HQ, HK, D, R, dtype, weights)
    pos = first + np.tile(np.arange(T), (B, 1))
    kw = dict(l2=l2, interleaved=inter, eps=1e-5, out_dtype=ot)
    at = None if first == 0 else dev(pos, torch.int32)
    args = (dev(a["q"], it), dev(a["k"], it), dev(w[0]), dev(w[1]), dev(freq), at)
    out = cuda_lib.qk_norm_fwd(*args, **kw)
    got = cuda_lib.qk_norm_bwd(*args, dev(gy[0], it), dev(gy[1], it), **kw)
    for i, n in enumerate("qk"):
        rows = lambda m: m.reshape((B * T,) + m.shape[2:])  # noqa: E731
        x, wn = rows(a[n]), w[i]
        ref = do.norm_fwd(x, wn, freq, pos.ravel(), l2, inter, 1e-5).reshape(a[n].shape)
        close(n + "_out", out[i], ref)
        dx, dw = do.norm_bwd(x, wn, freq, pos.ravel(), rows(gy[i]), l2, inter, 1e-5)
        # dx = r (g w - xhat mean(g w xhat)): with one column the two cancel but for
        # eps / x^2 of them, and four roundings of 2^-24 of the terms stay
        r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / (1 if l2 else D) + 1e-5)
        terms = np.abs(r * rows(gy[i])).max() * (1.0 if wn is None else np.abs(wn).max())
        d = np.abs(got["d" + n].double().cpu().numpy() - dx.reshape(a[n].shape))
        if d.max() > 2.0 ** -22 * terms:
            close("d" + n, got["d" + n], dx.reshape(a[n].shape))
        if weights:
            close("dw_" + n, got["dw_" + n], dw)
    assert ("dw_q" in got) == weights


@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 64), ("f32", 74, 74), ("bf16", 64, 0)])
def test_qk_norm_of_one_token_and_column_ranges(cuda_lib, dtype, D, R):
    """A token a row at its own position, in column ranges at several alignments, is what
    the same token is in a sequence."""
    import torch
    a, w, freq, gy, it, ot = qk_case((4, 30), 4, 2, D, R, dtype, True)
    q, k, f = dev(a["q"], it), dev(a["k"], it), dev(freq)
    w_q, w_k = dev(w[0]), dev(w[1])
    whole = cuda_lib.qk_norm_fwd(q, k, w_q, w_k, f)
    at = torch.tensor([29, 0, 7, 12], dtype=torch.int32, device="cuda")
    rows = torch.arange(4, device="cuda")
    for shift in (0, 1, 8):
        wide = torch.full((4, shift + 6 * D + 5), float("nan"), dtype=it, device="cuda")
        wide[:, shift:shift + 4 * D] = q[rows, at.long()].flatten(1)
        wide[:, shift + 4 * D:shift + 6 * D] = k[rows, at.long()].flatten(1)
        q1 = wide[:, shift:shift + 4 * D].unflatten(-1, (4, D))
        k1 = wide[:, shift + 4 * D:shift + 6 * D].unflatten(-1, (2, D))
        got = cuda_lib.qk_norm_fwd(q1, k1, w_q, w_k, f, at if R else None)
        for g, m in zip(got, whole):
            # one instance sums a row in another order than the other: an ulp or two
            d = (g.double() - m[rows, at.long()].double()).abs()
            assert float(d.max()) <= (2.0 ** -8 if dtype == "bf16" else 1e-6) * float(m.abs().max())


def test_qk_norm_zero_rows_and_one_weight(cuda_lib):
    import torch
    a, w, freq, gy, it, ot = qk_case((1, 6), 2, 2, 32, 16, "f32", True)
    a["q"][0, 3] = 0.0
    q, k, f = dev(a["q"]), dev(a["k"]), dev(freq)
    g = cuda_lib.qk_norm_bwd(q, k, dev(w[0]), None, f, None, dev(gy[0]), dev(gy[1]))
    assert "dw_q" in g and "dw_k" not in g
    out = cuda_lib.qk_norm_fwd(q, k, dev(w[0]), None, f)
    assert not out[0][0, 3].any() and bool(out[0].isfinite().all())
    dx, dw = do.norm_bwd(a["q"][0], w[0], freq, np.arange(6), gy[0][0])
    close("dq", g["dq"], dx[None])
    close("dw_q", g["dw_q"], dw)
    dx, _ = do.norm_bwd(a["k"][0], None, freq, np.arange(6), gy[1][0])
    close("dk", g["dk"], dx[None])


def test_qk_norm_past_32_bits(cuda_lib):
    """Batch rows further apart than 2^31 elements."""
    import torch
    apart = (1 << 31) + 128
    big = torch.empty(apart + 8 * 256, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((2, 8, 2, 128), (apart, 256, 128, 1))
    q.normal_()
    k = q[:, :, :1].contiguous()
    dense = q.contiguous()
    f = torch.ones(64, device="cuda")
    want, got = cuda_lib.qk_norm_fwd(dense, k, freq=f), cuda_lib.qk_norm_fwd(q, k, freq=f)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    g1 = cuda_lib.qk_norm_bwd(dense, k, None, None, f, None, want[0], want[1])
    g2 = cuda_lib.qk_norm_bwd(q, k, None, None, f, None, want[0], want[1])
    assert torch.equal(g1["dq"], g2["dq"]) and torch.equal(g1["dk"], g2["dk"])


# ------------------------------------------------------- a layer of them all

def test_a_layer_of_them_trains_and_decodes(cuda_lib):
    """Convolution, unit keys and turned queries, the delta rule and the gated norm as a
    layer runs them: the last tokens of sequences decoded one by one from the prompt's states
    get the outputs of a full pass.  fp32; the parts' errors of 1e-6 each, five in a row and
    the norm's 1 / rms of up to 3 between them: 1e-4 of the largest leaves a factor of 6."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    B, T, H, G, P, N, new = 3, 90, 4, 2, 16, 32, 6
    ch = 2 * G * N + H * P
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    u, z, dt, beta = n(B, T, ch), n(B, T, H * P), n(B, T, H) - 2, n(B, T, H)
    w, bias, norm = 0.5 * n(ch, 4), 0.1 * n(ch), 1 + 0.1 * n(H * P)
    dt_bias, A = 0.1 * n(H), -torch.exp(0.3 * n(H))
    freq = torch.tensor([1.0, 0.5, 0.2, 0.1], device="cuda")

    def split(x):
        q, k, v = x.split([G * N, G * N, H * P], -1)
        return q.unflatten(-1, (G, N)), k.unflatten(-1, (G, N)), v.unflatten(-1, (H, P))

    def prompt(m):
        x, conv = cuda_lib.causal_conv_fwd(u[:, :m].contiguous(), w, bias)
        q, k, v = split(x)
        q, k = cuda_lib.qk_norm_fwd(q, k, freq=freq, l2=True)
        y, S = cuda_lib.gated_delta_fwd(q, k, v, dt[:, :m].contiguous(), dt_bias, A,
                                        beta[:, :m].contiguous(), scale=N ** -0.5)
        out = cuda_lib.gated_norm_fwd(y.flatten(-2), z[:, :m].contiguous(), norm, H * P)[0]
        return out, conv, S
    full, conv_all, S_all = prompt(T)
    _, conv, S = prompt(T - new)
    for i in range(T - new, T):
        x = cuda_lib.causal_conv_step(u[:, i].contiguous(), conv, w, bias)
        q, k, v = split(x)
        at = torch.full((B,), i, dtype=torch.int32, device="cuda")
        q, k = cuda_lib.qk_norm_fwd(q, k, freq=freq, positions=at, l2=True)
        y = cuda_lib.gated_delta_step(q, k, v, dt[:, i].contiguous(), dt_bias, A, beta[:, i].contiguous(),
                                      S, scale=N ** -0.5)
        out = cuda_lib.gated_norm_fwd(y.flatten(-2), z[:, i].contiguous(), norm, H * P)[0]
        assert float((out - full[:, i]).abs().max()) <= 1e-4 * float(full.abs().max())
    assert float((S - S_all).abs().max()) <= 1e-4 * float(S_all.abs().max())


def test_calls_of_two_threads(cuda_lib):
    """Two host threads at the same time, each with shapes and a stream of its own: the bits
    of the same calls one after another (sizes whose shared memory differs)."""
    import threading

    import torch
    jobs = []
    for i, (case, D) in enumerate([((2, 190, 6, 3, 128, 128, "bf16", True, None), 1024),
                                   ((1, 1100, 2, 1, 24, 40, "f32", True, [1001]), 700)]):
        it, _ = types(case[6])
        a, init, dy, _, ln = delta_case(*case)
        x, more = on_gpu(a, it), dict(init_states=dev(init), lengths=dev(ln, torch.int32))
        g = np.random.default_rng(i)
        q, k, dq, dk = (dev(g.standard_normal((3, 20, 2, D)), it) for _ in range(4))
        w, f = dev(g.standard_normal(D), torch.float32), dev(g.random(D // 4), torch.float32)

        def run(x=x, more=more, dy=dev(dy, it), q=q, k=k, w=w, f=f, dq=dq, dk=dk):
            b = cuda_lib.gated_delta_bwd(*x, dy, **more)
            n = cuda_lib.qk_norm_bwd(q, k, w, w, f, None, dq, dk)
            return [*cuda_lib.gated_delta_fwd(*x, **more), *b.values(), *n.values()]
        jobs.append(run)
    want = [[t.clone() for t in run()] for run in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(run, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = run()
                    torch.cuda.current_stream().synchronize()
                    wrong.extend(not torch.equal(a, b) for a, b in zip(got, ref))
        except Exception as e:  # noqa: BLE001 - handed to the test's own thread
            wrong.append(e)
    threads = [threading.Thread(target=work, args=z) for z in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(wrong) == 20 * sum(len(w) for w in want) and not any(wrong), [w for w in wrong if w][:3]
