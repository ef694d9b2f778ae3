"""The layer operators (causal convolution, selective scan, single-token steps,
block norm) against the fp64 oracle (``oracle/layer_ops.py``) on a GPU.

Tolerances.  Inputs are rounded to their storage type first, so the oracle
sees the kernels' values and what is left is the kernels' own fp32 arithmetic:
a few roundings of 6e-8 per operation, exponentials, softplus and sigmoid good
to ~5e-7, and sums whose terms' errors are independent.  20 such errors in a
row are 1e-5, so fp32 results lie within 1e-5 in relative L2 and 4e-5 of the
largest value anywhere.  A bf16 output has one more rounding, half a unit in
the 8th bit: 2^-8 of the value."""
import numpy as np
import pytest

from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu


def stored(a, dtype):
    """a as the kernels read it, in fp64."""
    import torch
    return None if a is None else torch.from_numpy(np.asarray(a)).to(dtype).double().numpy()


def dev(a, dtype=None):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(
        "cuda", dtype or torch.float32)


def close(name, got, ref):
    import torch
    assert got.shape == ref.shape, name
    if got.numel() == 0:
        return
    bf = got.dtype == torch.bfloat16
    g = got.detach().double().cpu().numpy()
    assert np.isfinite(g).all(), name
    d, top = np.abs(g - ref), np.abs(ref).max()
    bound = 4e-5 * top + (2.0 ** -8 * np.abs(ref) if bf else 0.0)
    assert np.all(d <= bound + 1e-30), (name, float((d - bound).max()), float(top))
    if not bf:
        assert np.linalg.norm(g - ref) <= 1e-5 * np.linalg.norm(ref) + 1e-30, name


def types(dtype):
    import torch
    return {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
            "mixed": (torch.bfloat16, torch.float32)}[dtype]


# ---------------------------------------------------------------- convolution

CONV = [
    # B, T, C, K, dtype, bias, init, lengths, silu
    (1, 1, 8, 4, "bf16", True, False, None, True),
    (1, 1, 1, 2, "f32", False, True, None, False),
    (2, 2, 24, 4, "f32", True, True, [2, 1], True),          # shorter than the window
    (3, 37, 64, 4, "bf16", True, False, [37, 0, 1], True),    # an empty row
    (2, 300, 40, 3, "mixed", False, True, None, True),
    (2, 129, 33, 2, "bf16", True, True, [128, 77], False),    # no vector fits
    (1, 1000, 257, 4, "f32", True, False, None, True),
    (4, 70, 520, 4, "bf16", True, True, [3, 70, 2, 64], True),
]


@pytest.mark.parametrize("case", CONV)
def test_conv_matches_oracle(cuda_lib, case):
    import torch
    B, T, C, K, dtype, has_bias, has_init, lengths, silu = case
    it, ot = types(dtype)
    g = np.random.default_rng(B * 1000 + T + C)
    x, dy = stored(g.standard_normal((B, T, C)), it), stored(g.standard_normal((B, T, C)), it)
    w = stored(g.uniform(-0.5, 0.5, (C, K)), torch.float32)
    bias = stored(g.standard_normal(C), torch.float32) if has_bias else None
    init = stored(g.standard_normal((B, K - 1, C)), it) if has_init else None
    df = stored(g.standard_normal((B, K - 1, C)), it)
    ln = dev(np.array(lengths), torch.int32) if lengths else None
    a = (dev(x, it), dev(w), dev(bias))
    y, fin = cuda_lib.causal_conv_fwd(*a, init_state=dev(init, it), lengths=ln, silu=silu,
                                      out_dtype=ot)
    yr, fr = lo.conv_fwd(x, w, bias, init, lengths, silu)
    close("y", y, yr)
    assert np.array_equal(fin.double().cpu().numpy(), fr)
    r = lo.conv_bwd(x, w, bias, dy, init, lengths, silu, df)
    out = cuda_lib.causal_conv_bwd(*a, dev(dy, it), init_state=dev(init, it), lengths=ln, silu=silu,
                                   dfinal_state=dev(df, it), out_dtype=ot)
    for k, v in out.items():
        close(k, v, r[k])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), "lowest"])
@pytest.mark.parametrize("C,dtype", [(33, "bf16"), (64, "bf16"), (48, "f32"), (7, "f32")])
def test_conv_padding_reaches_nothing(cuda_lib, C, dtype, value):
    import torch
    it, _ = types(dtype)
    value = torch.finfo(it).min if value == "lowest" else value
    g, T, lengths = np.random.default_rng(C), 150, [150, 0, 77, 1]
    x, dy = (dev(g.standard_normal((4, T, C)), it) for _ in range(2))
    w, init = dev(g.standard_normal((C, 4))), dev(g.standard_normal((4, 3, C)), it)
    ln = dev(np.array(lengths), torch.int32)

    def run(fill):
        xp, dp = padded(x, lengths, fill), padded(dy, lengths, fill)
        got = cuda_lib.causal_conv_bwd(xp, w, None, dp, init_state=init, lengths=ln)
        got["y"], got["final"] = cuda_lib.causal_conv_fwd(xp, w, None, init_state=init, lengths=ln)
        return got

    zero, other = run(0.0), run(value)
    assert all(torch.equal(zero[k], other[k]) for k in zero)
    assert all(bool(torch.isfinite(v).all()) for v in other.values())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_rows_of_a_decoding_step_reach_nothing(cuda_lib, dtype):
    """Rows without a slot may hold anything: outputs 0, and no state is touched."""
    import torch
    it, _ = types(dtype)
    g, nan = np.random.default_rng(3), float("nan")
    slots = dev(np.array([2, -1, 0, 9, -7]), torch.int32)  # 9 is past the 4 states
    live = [0, 2]

    def rows(*shape):
        t = dev(g.standard_normal((5,) + shape), it)
        t[[1, 3, 4]] = nan
        return t

    def check(y, state, before):
        assert bool((y[[1, 3, 4]] == 0).all()) and bool(torch.isfinite(y[live]).all())
        assert torch.equal(state[[1, 3]], before[[1, 3]]) and bool(torch.isfinite(state).all())

    A = dev(-np.exp(g.standard_normal((24, 16))))
    state = dev(g.standard_normal((4, 24, 16)))
    before = state.clone()
    y = cuda_lib.selective_step(rows(24), rows(24), None, A, rows(1, 16), rows(1, 16), state,
                                z=rows(24), slots=slots)
    check(y, state, before)
    state = dev(g.standard_normal((4, 3, 8, 16)))
    before = state.clone()
    y = cuda_lib.ssd_step(rows(3, 8), rows(3), None, A[0, :3].contiguous(), rows(1, 16),
                          rows(1, 16), state, slots=slots)
    check(y, state, before)
    state = dev(g.standard_normal((4, 3, 24)), it)
    before = state.clone()
    y = cuda_lib.causal_conv_step(rows(24), state, dev(g.standard_normal((24, 4))), slots=slots)
    check(y, state, before)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_backward_under_load(cuda_lib, dtype):
    """At a size that keeps the memory system busy, where a copy read before it has
    arrived would show: the gradients against the formula in fp64, call after call
    with the same bits."""
    import torch
    it, _ = types(dtype)
    B, T, C, K = 4, 4096, 1792, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(B, T, C, generator=g, device="cuda").to(it) for _ in range(2))
    w, bias = torch.randn(C, K, generator=g, device="cuda") * 0.5, torch.zeros(C, device="cuda")
    first = {k: v.clone() for k, v in cuda_lib.causal_conv_bwd(x, w, bias, dy).items()}
    xp = torch.nn.functional.pad(x.double(), (0, 0, K - 1, 0))
    u = sum(xp[:, k:k + T] * w[:, k].double() for k in range(K))
    sg = torch.sigmoid(u)
    du = dy.double() * sg * (1 + u * (1 - sg))
    dup = torch.nn.functional.pad(du, (0, 0, 0, K - 1))
    dx = sum(dup[:, K - 1 - k:K - 1 - k + T] * w[:, k].double() for k in range(K))
    close("dx", first["dx"], dx.cpu().numpy())
    close("dw", first["dw"], torch.stack([(du * xp[:, k:k + T]).sum((0, 1)) for k in range(K)],
                                         1).cpu().numpy())
    close("dbias", first["dbias"], du.sum((0, 1)).cpu().numpy())
    junk = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(50):
        junk.add_(1)  # x and dy leave the L2 cache
        again = cuda_lib.causal_conv_bwd(x, w, bias, dy)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_conv_of_a_column_range_and_in_place_step(cuda_lib):
    """x as columns of a wider tensor, at an offset that allows 8-byte accesses
    only; then tokens one by one from the prompt's state."""
    import torch
    g = np.random.default_rng(0)
    B, T, C, K, W = 3, 21, 40, 4, 100
    wide = dev(g.standard_normal((B, T, W)), torch.bfloat16)
    x = wide[..., 4:4 + C]
    w, bias = dev(g.uniform(-0.5, 0.5, (C, K))), dev(g.standard_normal(C))
    y, fin = cuda_lib.causal_conv_fwd(x, w, bias)
    y2, fin2 = cuda_lib.causal_conv_fwd(x.contiguous(), w, bias)
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    dy = dev(g.standard_normal((B, T, C)), torch.bfloat16)
    a, b = (cuda_lib.causal_conv_bwd(v, w, bias, dy) for v in (x, x.contiguous()))
    assert all(torch.equal(a[k], b[k]) for k in a)
    # prompt of 18, then 3 tokens, rows in permuted slots
    state = torch.full((5, K - 1, C), 7.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    _, f = cuda_lib.causal_conv_fwd(x[:, :18], w, bias)
    state[slots.long()] = f
    for t in range(18, T):
        yt = cuda_lib.causal_conv_step(x[:, t], state, w, bias, slots=slots)
        assert torch.equal(yt, y[:, t])
    assert torch.equal(state[slots.long()], fin)
    assert bool((state[[1, 3]] == 7.0).all())


def test_conv_states_side_by_side(cuda_lib):
    """The initial and the final state next to each other in one buffer are fine; one for
    both, or shifted into each other, is refused."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(8)
    x, w = torch.randn(2, 9, 8, generator=g, device="cuda"), torch.randn(8, 4, generator=g, device="cuda")
    buf = torch.randn(3, 2, 3, 8, generator=g, device="cuda")
    init = buf[1].clone()
    y, fin = cuda_lib.causal_conv_fwd(x, w, init_state=init)
    for k in (0, 2):
        y2, fin2 = cuda_lib.causal_conv_fwd(x, w, init_state=buf[1], final_state=buf[k])
        assert torch.equal(y2, y) and torch.equal(buf[k], fin) and torch.equal(buf[1], init)
    flat = buf.view(-1)
    for at in (48, 49, 95, 1):
        with pytest.raises(cuda_lib.SSDError) as e:
            cuda_lib.causal_conv_fwd(x, w, init_state=buf[1], final_state=flat[at:at + 48].view(2, 3, 8))
        assert e.value.status == 1


# ------------------------------------------------------------- selective scan

def scan_inputs(seed, B, T, D, N, G, it, gated, has_init):
    import torch
    f32 = torch.float32
    g = np.random.default_rng(seed)
    step = np.exp(g.uniform(np.log(1e-3), np.log(0.2), (B, T, D)))
    bias = np.log(np.expm1(np.exp(g.uniform(np.log(1e-3), np.log(0.1), D))))
    a = dict(x=stored(g.standard_normal((B, T, D)), it),
             dt=stored(np.log(np.expm1(step)) - bias, it), dt_bias=stored(bias, f32),
             A=stored(-(1.0 + np.arange(N)) * np.exp(g.uniform(-0.3, 0.3, (D, N))), f32),
             B=stored(g.standard_normal((B, T, G, N)), it),
             C=stored(g.standard_normal((B, T, G, N)), it), D=stored(g.uniform(0, 1, D), f32),
             z=stored(g.standard_normal((B, T, D)), it) if gated else None)
    init = stored(g.standard_normal((B, D, N)), f32) if has_init else None
    return a, init, g


def scan_dev(a, it):
    return [dev(a[k], it if k in ("x", "dt", "B", "C", "z") else None)
            for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")]


SCAN = [
    # B, T, D, N, G, dtype, gated, init, lengths
    (1, 1, 1, 1, 1, "f32", False, False, None),
    (1, 1, 32, 16, 1, "bf16", True, True, None),
    (2, 31, 64, 16, 1, "f32", True, True, [31, 7]),
    (3, 33, 70, 16, 2, "bf16", True, False, [33, 0, 1]),      # an empty row, ragged groups
    (2, 97, 6, 8, 3, "f32", False, True, None),               # two channels a group
    (1, 700, 40, 5, 1, "f32", True, False, None),             # several chunks forward
    (2, 200, 130, 24, 1, "mixed", True, True, [150, 200]),
    (1, 130, 33, 64, 1, "f32", False, True, [129]),
    (1, 64, 300, 33, 3, "bf16", True, True, None),
    (1, 3000, 16, 16, 1, "f32", True, True, None),            # a long walk over chunks
]


@pytest.mark.parametrize("case", SCAN)
def test_scan_matches_oracle(cuda_lib, case):
    import torch
    B, T, D, N, G, dtype, gated, has_init, lengths = case
    it, ot = types(dtype)
    a, init, g = scan_inputs(T * 7 + D + N, B, T, D, N, G, it, gated, has_init)
    dout = stored(g.standard_normal((B, T, D)), it)
    df = stored(g.standard_normal((B, D, N)), torch.float32)
    ln = dev(np.array(lengths), torch.int32) if lengths else None
    args = scan_dev(a, it)
    out, fin = cuda_lib.selective_scan_fwd(*args, init_states=dev(init), lengths=ln, out_dtype=ot)
    orf, fr = lo.scan_fwd(init=init, lengths=lengths, **a)
    close("out", out, orf)
    close("final", fin, fr)
    r = lo.scan_bwd(*(a[k] for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")), dout, init,
                    lengths, df)
    got = cuda_lib.selective_scan_bwd(*args, dev(dout, it), init_states=dev(init), lengths=ln,
                                      dfinal_states=dev(df), out_dtype=ot)
    assert ("dz" in got) == gated and ("dinit_states" in got) == has_init
    for k, v in got.items():
        close(k, v, r[k])


def padded(t, lengths, value):
    """A copy of t (batch, seqlen, ..) with value from each row's length on."""
    t = t.clone()
    for b, n in enumerate(lengths):
        t[b, n:] = value
    return t


@pytest.mark.parametrize("value", [float("nan"), float("inf"), "lowest"])
@pytest.mark.parametrize("T,D,N,dtype", [(70, 37, 16, "bf16"), (700, 64, 16, "bf16"),
                                         (333, 30, 24, "f32")])
def test_scan_padding_reaches_nothing(cuda_lib, T, D, N, dtype, value):
    """Padded positions may hold anything: every output has the bits of zero padding."""
    import torch
    it, _ = types(dtype)
    value = torch.finfo(it).min if value == "lowest" else value
    lengths = [T, 0, T // 2 + 1, 1]
    a, init, g = scan_inputs(T + D, 4, T, D, N, 1, it, True, True)
    dout = dev(g.standard_normal((4, T, D)), it)
    ln = dev(np.array(lengths), torch.int32)

    def run(fill):
        args = [padded(t, lengths, fill) if k in ("x", "dt", "B", "C", "z") else t
                for k, t in zip(("x", "dt", "dt_bias", "A", "B", "C", "D", "z"), scan_dev(a, it))]
        got = cuda_lib.selective_scan_bwd(*args, padded(dout, lengths, fill), init_states=dev(init),
                                          lengths=ln)
        got["out"], got["final"] = cuda_lib.selective_scan_fwd(*args, init_states=dev(init), lengths=ln)
        return got

    zero, other = run(0.0), run(value)
    assert all(torch.equal(zero[k], other[k]) for k in zero)
    assert all(bool(torch.isfinite(v).all()) for v in other.values())


def test_scan_without_bias_skip_or_final_gradient(cuda_lib):
    import torch
    a, _, g = scan_inputs(5, 2, 40, 32, 16, 1, torch.float32, False, False)
    dout = g.standard_normal((2, 40, 32)).astype(np.float32)
    x, dt, _, A, B, C, _, _ = scan_dev(a, torch.float32)
    b = {**a, "dt_bias": None, "D": None}
    out, none = cuda_lib.selective_scan_fwd(x, dt, None, A, B, C, return_final_states=False)
    assert none is None
    close("out", out, lo.scan_fwd(**b)[0])
    r = lo.scan_bwd(b["x"], b["dt"], None, b["A"], b["B"], b["C"], None, None, dout)
    got = cuda_lib.selective_scan_bwd(x, dt, None, A, B, C, None, None, dev(dout))
    for k, v in got.items():
        close(k, v, r[k])


def test_scan_large_steps_stay_finite(cuda_lib):
    """Steps past softplus's linear branch and decays that underflow to 0: the
    state forgets at once; nothing overflows."""
    import torch
    a, init, g = scan_inputs(9, 1, 50, 32, 16, 1, torch.float32, True, True)
    a["dt"] = stored(g.choice([-80.0, 0.0, 30.0, 60.0], (1, 50, 32)), torch.float32)
    dout = stored(g.standard_normal((1, 50, 32)), torch.float32)
    args = scan_dev(a, torch.float32)
    out, fin = cuda_lib.selective_scan_fwd(*args, init_states=dev(init))
    orf, fr = lo.scan_fwd(init=init, **a)
    close("out", out, orf)
    close("final", fin, fr)
    r = lo.scan_bwd(*(a[k] for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")), dout, init)
    got = cuda_lib.selective_scan_bwd(*args, dev(dout), init_states=dev(init))
    for k, v in got.items():
        close(k, v, r[k])


def test_scan_gradients_are_differences(cuda_lib):
    """The kernels' gradients along a random direction against the fp64 oracle's
    central difference of the loss."""
    import torch
    a, init, g = scan_inputs(11, 2, 45, 24, 16, 1, torch.float32, True, True)
    dout = g.standard_normal((2, 45, 24)).astype(np.float32).astype(np.float64)
    got = cuda_lib.selective_scan_bwd(*scan_dev(a, torch.float32), dev(dout), init_states=dev(init))

    def loss(**kw):
        b = {**a, "init": init, **kw}
        return float((lo.scan_fwd(**b)[0] * dout).sum())
    for k, gk in (("x", "dx"), ("dt", "ddt"), ("dt_bias", "ddt_bias"), ("A", "dA"), ("B", "dB"),
                  ("C", "dC"), ("D", "dD"), ("z", "dz"), ("init", "dinit_states")):
        base = init if k == "init" else a[k]
        v = g.standard_normal(base.shape)
        want = (loss(**{k: base + 1e-6 * v}) - loss(**{k: base - 1e-6 * v})) / 2e-6
        mine = got[gk].double().cpu().numpy()
        assert abs((mine * v).sum() - want) <= 1e-5 * np.linalg.norm(mine) * np.linalg.norm(v), k


def test_scan_of_column_ranges(cuda_lib):
    import torch
    it = torch.bfloat16
    a, init, g = scan_inputs(13, 2, 50, 48, 16, 1, it, True, False)
    x, dt, bias, A, B, C, D, z = scan_dev(a, it)
    bc = torch.cat([torch.zeros(2, 50, 5, dtype=it, device="cuda"), B[:, :, 0], C[:, :, 0]], 2)
    zw = torch.cat([z, x], 2)
    v = (x, dt, bias, A, bc[..., 5:21].unsqueeze(2), bc[..., 21:].unsqueeze(2), D, zw[..., :48])
    o1, f1 = cuda_lib.selective_scan_fwd(x, dt, bias, A, B, C, D, z)
    o2, f2 = cuda_lib.selective_scan_fwd(*v)
    assert torch.equal(o1, o2) and torch.equal(f1, f2)
    dout = dev(g.standard_normal((2, 50, 48)), it)
    g1 = cuda_lib.selective_scan_bwd(x, dt, bias, A, B, C, D, z, dout)
    g2 = cuda_lib.selective_scan_bwd(*v, dout)
    assert all(torch.equal(g1[k], g2[k]) for k in g1)


@pytest.mark.parametrize("T,D,G", [(50, 37, 1), (333, 48, 1), (41, 66, 2), (1, 5, 1)])
@pytest.mark.parametrize("at", [0, 1, 4, "end"])
def test_scan_of_odd_column_ranges(cuda_lib, T, D, G, at):
    """z at odd and even columns of a wider tensor of odd rows, and as its very last
    columns (the whole words that cover a row must not pass the tensor's ends), B and C at
    odd columns; everything beside them is NaN."""
    import torch
    it = torch.bfloat16
    a, init, g = scan_inputs(T + D, 3, T, D, 16, G, it, True, True)
    x, dt, bias, A, B, C, Dv, z = scan_dev(a, it)
    W = 2 * D + (2 * D + 1) % 2  # odd
    off = W - D if at == "end" else at
    zw = torch.full((3, T, W), float("nan"), dtype=it, device="cuda")
    zw[..., off:off + D] = z
    bc = torch.full((3, T, 2 * G * 16 + 1), float("nan"), dtype=it, device="cuda")
    bc[..., 1:] = torch.cat([B.flatten(2), C.flatten(2)], 2)
    Bw, Cw = (t.unflatten(2, (G, 16)) for t in bc[..., 1:].split(G * 16, 2))
    v = (x, dt, bias, A, Bw, Cw, Dv, zw[..., off:off + D])
    out, fin = cuda_lib.selective_scan_fwd(*v, init_states=dev(init))
    orf, fr = lo.scan_fwd(init=init, **a)
    close("out", out, orf)
    close("final", fin, fr)
    dout = stored(g.standard_normal((3, T, D)), it)
    r = lo.scan_bwd(*(a[k] for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")), dout, init)
    for k, t in cuda_lib.selective_scan_bwd(*v, dev(dout, it), init_states=dev(init)).items():
        close(k, t, r[k])


def test_repeats_under_load_are_bit_identical(cuda_lib):
    """As test_conv_backward_under_load, for the rings of the scan and of the block
    norm: their values are pinned at small sizes, a late copy would change bits."""
    import torch
    it, g = torch.bfloat16, torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    B, T, D, N = 2, 2048, 1536, 16
    A = -torch.arange(1.0, N + 1, device="cuda").repeat(D, 1)
    x, z, dout = (r(B, T, D).to(it) for _ in range(3))
    sc = (x, (r(B, T, D) - 4).to(it), r(D), A, r(B, T, 1, N).to(it), r(B, T, 1, N).to(it), r(D), z)
    bn = (r(8192, 4096), r(8192, 4096).to(it), r(4096), r(4096), r(2, 4096))
    dh, w = r(8192, 4096).to(it), r(D, 4)
    calls = (lambda: dict(enumerate(cuda_lib.selective_scan_fwd(*sc))),
             lambda: cuda_lib.selective_scan_bwd(*sc, dout),
             lambda: dict(enumerate(cuda_lib.block_norm_fwd(*bn))),
             lambda: cuda_lib.block_norm_bwd(*bn, dh, bn[0]),
             lambda: dict(enumerate(cuda_lib.causal_conv_fwd(x, w))))
    junk = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for call in calls:
        first = {k: v.clone() for k, v in call().items()}
        for _ in range(15):
            junk.add_(1)  # the inputs leave the L2 cache
            assert all(torch.equal(first[k], v) for k, v in call().items())


def test_repeated_calls_are_bit_identical(cuda_lib):
    import torch
    a, init, g = scan_inputs(17, 2, 500, 200, 16, 1, torch.bfloat16, True, True)
    args, dout = scan_dev(a, torch.bfloat16), dev(g.standard_normal((2, 500, 200)), torch.bfloat16)
    r1, r2 = (cuda_lib.selective_scan_bwd(*args, dout, init_states=dev(init)) for _ in range(2))
    assert all(torch.equal(r1[k], r2[k]) for k in r1)
    w = dev(g.standard_normal((200, 4)))
    r1, r2 = (cuda_lib.causal_conv_bwd(args[0], w, None, dout) for _ in range(2))
    assert all(torch.equal(r1[k], r2[k]) for k in r1)


# ---------------------------------------------------------------- single tokens

@pytest.mark.parametrize("B,D,N,G,dtype,gated", [
    (1, 1, 1, 1, "f32", False), (3, 64, 16, 1, "bf16", True), (5, 33, 16, 3, "mixed", True),
    (2, 70, 7, 1, "f32", True), (4, 40, 64, 2, "bf16", False), (2, 24, 200, 1, "f32", True),
    (64, 1536, 16, 1, "bf16", True)])
def test_selective_step_matches_oracle(cuda_lib, B, D, N, G, dtype, gated):
    import torch
    it, ot = types(dtype)
    a, _, g = scan_inputs(B + D + N, B, 1, D, N, G, it, gated, False)
    n = B + 3
    slots = g.permutation(n)[:B]
    state = stored(g.standard_normal((n, D, N)), torch.float32)
    sd = dev(state)
    args = [t[:, 0] if t is not None and t.dim() > 2 else t for t in scan_dev(a, it)]
    y = cuda_lib.selective_step(*args[:6], sd, *args[6:], slots=dev(slots, torch.int32), out_dtype=ot)
    orf, fr = lo.scan_fwd(init=state[slots], **a)
    close("y", y, orf[:, 0])
    want = state.copy()
    want[slots] = fr
    close("state", sd, want)
    rest = np.setdiff1d(np.arange(n), slots)
    assert np.array_equal(sd.cpu().numpy()[rest], state[rest].astype(np.float32))


@pytest.mark.parametrize("B,C,K,dtype,has_bias,silu", [
    (1, 1, 2, "f32", False, True), (3, 24, 2, "bf16", True, True), (5, 33, 3, "mixed", True, True),
    (2, 777, 3, "f32", True, False), (7, 41, 4, "mixed", False, True), (3, 40, 3, "bf16", True, False),
    (4, 36, 2, "mixed", True, True), (2, 1023, 4, "bf16", True, True), (64, 1792, 4, "bf16", True, True)])
def test_conv_step_matches_oracle(cuda_lib, B, C, K, dtype, has_bias, silu):
    import torch
    it, ot = types(dtype)
    g = np.random.default_rng(B + C + K)
    x, n = stored(g.standard_normal((B, C)), it), B + 2
    w = stored(g.uniform(-0.5, 0.5, (C, K)), torch.float32)
    bias = stored(g.standard_normal(C), torch.float32) if has_bias else None
    slots = g.permutation(n)[:B]
    state = stored(g.standard_normal((n, K - 1, C)), it)
    yr, fr = lo.conv_fwd(x[:, None], w, bias, state[slots], None, silu)
    want = state.copy()
    want[slots] = fr
    wide = torch.zeros(B, C + 5, dtype=it, device="cuda")
    wide[:, 3:3 + C] = dev(x, it)
    for xd in (dev(x, it), wide[:, 3:3 + C]):  # dense, and columns at an odd offset
        sd = dev(state, it)
        y = cuda_lib.causal_conv_step(xd, sd, dev(w), dev(bias), slots=dev(slots, torch.int32),
                                      silu=silu, out_dtype=ot)
        close("y", y, yr[:, 0])
        assert np.array_equal(sd.double().cpu().numpy(), want)


@pytest.mark.parametrize("D,N,G,dtype", [(48, 16, 1, "bf16"), (37, 7, 1, "bf16"), (66, 16, 2, "mixed"),
                                         (33, 16, 3, "f32")])
def test_selective_step_of_column_ranges(cuda_lib, D, N, G, dtype):
    """z, B and C as columns of wider rows, at odd and even offsets: the bits of dense ones."""
    import torch
    it, ot = types(dtype)
    g = np.random.default_rng(D)
    r = lambda *s: dev(g.standard_normal(s), it)  # noqa: E731
    x, dt, z, B, C = r(5, D), r(5, D), r(5, D), r(5, G, N), r(5, G, N)
    A, state = dev(-np.exp(g.standard_normal((D, N)))), dev(g.standard_normal((5, D, N)))
    for at in (0, 1, 2, 5):
        wide = r(5, at + D + 2 * G * N + 1)
        zw, Bw, Cw = (wide[:, a:a + n] for a, n in ((at, D), (at + D, G * N), (at + D + G * N, G * N)))
        for t, v in ((zw, z), (Bw, B), (Cw, C)):
            t.copy_(v.reshape(t.shape))
        s1, s2 = state.clone(), state.clone()
        y1 = cuda_lib.selective_step(x, dt, None, A, B, C, s1, None, z, out_dtype=ot)
        y2 = cuda_lib.selective_step(x, dt, None, A, Bw.unflatten(1, (G, N)), Cw.unflatten(1, (G, N)),
                                     s2, None, zw, out_dtype=ot)
        assert torch.equal(y1, y2) and torch.equal(s1, s2)


def test_softplus_within_its_bound(cuda_lib):
    """With x = B = C = 1 and a state of 0 the output is delta itself.  v log2(e) has two
    roundings, 1e-7 of v together, which e^v makes errors of its value; 2^v, the
    quotient and the logarithm's series add 5e-7."""
    import torch
    v = stored(np.linspace(-86.0, 40.0, 20001), torch.float32)
    want = np.logaddexp(0.0, v)
    n = len(v)
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    A, dt = -one(n, 1), dev(v)
    got = [cuda_lib.selective_scan_fwd(one(1, 1, n), dt.view(1, 1, n), None, A, one(1, 1, 1, 1),
                                       one(1, 1, 1, 1))[0],
           cuda_lib.selective_step(one(1, n), dt.view(1, n), None, A, one(1, 1, 1), one(1, 1, 1),
                                   0 * one(1, n, 1)),
           cuda_lib.ssd_step(one(n, 1, 1), dt.view(n, 1), None, -one(1), one(n, 1, 1), one(n, 1, 1),
                             0 * one(n, 1, 1, 1))]
    for y in got:
        err = np.abs(y.double().cpu().numpy().ravel() / want - 1.0)
        assert np.all(err <= 5e-7 + 1e-7 * np.maximum(-v, 0.0)), float(err.max())


@pytest.mark.parametrize("B,H,P,N,G,dtype", [
    (1, 1, 1, 1, 1, "f32"), (1, 24, 64, 128, 1, "bf16"), (3, 6, 40, 33, 2, "mixed"),
    (2, 5, 16, 16, 1, "f32"), (7, 4, 128, 64, 2, "bf16"), (2, 2, 64, 200, 1, "f32"),
    (70, 16, 64, 128, 8, "bf16")])
def test_ssd_step_matches_oracle(cuda_lib, B, H, P, N, G, dtype):
    import torch
    it, ot = types(dtype)
    f32 = torch.float32
    g = np.random.default_rng(B + H + P + N)
    x, dt = stored(g.standard_normal((B, H, P)), it), stored(g.standard_normal((B, H)) - 2, it)
    bias, A = stored(g.standard_normal(H), f32), stored(-np.exp(g.uniform(0, 2.7, H)), f32)
    Bm, Cm = (stored(g.standard_normal((B, G, N)), it) for _ in range(2))
    D = stored(g.uniform(0, 1, H), f32)
    n = B + 2
    slots = g.permutation(n)[:B]
    state = stored(g.standard_normal((n, H, P, N)), f32)
    sd = dev(state)
    y = cuda_lib.ssd_step(dev(x, it), dev(dt, it), dev(bias), dev(A), dev(Bm, it), dev(Cm, it), sd,
                          dev(D), slots=dev(slots, torch.int32), out_dtype=ot)
    yr, fr = lo.ssd_step(x, dt, bias, A, Bm, Cm, D, state[slots])
    close("y", y, yr)
    want = state.copy()
    want[slots] = fr
    close("state", sd, want)


def test_empty_rows_touch_nothing(cuda_lib):
    """Negative and out-of-range slots: output 0, every state as it was."""
    import torch
    slots = torch.tensor([-1, 3, 9, 1], dtype=torch.int32, device="cuda")  # of 4 slots
    it = torch.bfloat16
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, w, state = r(4, 40).to(it), r(40, 4), r(4, 3, 40).to(it)
    before = state.clone()
    y = cuda_lib.causal_conv_step(x, state, w, slots=slots)
    assert bool((y[[0, 2]] == 0).all()) and bool((y[[1, 3]] != 0).any())
    assert torch.equal(state[[0, 2]], before[[0, 2]]) and not torch.equal(state[3], before[3])
    state = r(4, 40, 16)
    before = state.clone()
    bc = r(4, 1, 16).to(it)
    y = cuda_lib.selective_step(x, x, None, -torch.ones(40, 16, device="cuda"), bc, bc, state,
                                z=x, slots=slots)
    assert bool((y[[0, 2]] == 0).all()) and torch.equal(state[[0, 2]], before[[0, 2]])
    assert not torch.equal(state[1], before[1])
    state = r(4, 2, 20, 16)
    before = state.clone()
    y = cuda_lib.ssd_step(x.view(4, 2, 20), x[:, :2].contiguous(), None,
                          -torch.ones(2, device="cuda"), bc, bc, state, slots=slots)
    assert bool((y[[0, 2]] == 0).all()) and torch.equal(state[[0, 2]], before[[0, 2]])
    assert not torch.equal(state[3], before[3])


def test_steps_go_on_from_prompts(cuda_lib):
    """A prompt and then single tokens give what the whole sequence gives, for
    both scans (each within its own bar of the oracle)."""
    import torch
    f32 = torch.float32
    a, _, g = scan_inputs(21, 2, 40, 24, 16, 1, f32, True, False)
    args = scan_dev(a, f32)
    orf, fr = lo.scan_fwd(**a)
    cut = lambda t, s: t[:, s].contiguous() if t is not None and t.dim() > 2 else t  # noqa: E731
    _, state = cuda_lib.selective_scan_fwd(*(cut(t, slice(0, 35)) for t in args))
    for t in range(35, 40):
        v = [cut(q, t) for q in args]
        close("y", cuda_lib.selective_step(*v[:6], state, *v[6:]), orf[:, t])
    close("state", state, fr)


# ------------------------------------------------------------------ block norm

NORM = [
    # rows, F, in, residual, post, gates, scale
    (1, 3, "f32", "f32", True, 0, 1.0),
    (5, 64, "f32", "f32", True, 1, 0.5),
    (4, 8, "bf16", "f32", True, 4, 1.0),        # a gate row per row
    (700, 1536, "bf16", "f32", True, 2, 0.22),
    (301, 1001, "f32", "f32", False, 7, 1.0),   # odd width
    (64, 4096, "bf16", "bf16", True, 0, 1.0),
    (600, 520, "bf16", "bf16", False, 0, 2.0),
    (9, 8192, "f32", "f32", True, 3, 0.7),
    (6, 8191, "bf16", "f32", True, 2, 0.7),
    (2000, 24, "bf16", "f32", True, 8, 1.0),
    (1200, 100, "f32", "f32", True, 1200, 1.0),  # more gate rows than blocks
]


@pytest.mark.parametrize("case", NORM)
def test_block_norm_matches_oracle(cuda_lib, case):
    import torch
    rows, F, io, res, post, gates, scale = case
    it = torch.bfloat16 if io == "bf16" else torch.float32
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    f32 = torch.float32
    g = np.random.default_rng(rows + F)
    r, o = stored(g.standard_normal((rows, F)), rt), stored(g.standard_normal((rows, F)), it)
    wp, wq = stored(1 + 0.1 * g.standard_normal(F), f32), stored(1 + 0.1 * g.standard_normal(F), f32)
    wq = wq if post else None
    gate = stored(g.standard_normal((gates, F)), f32) if gates else None
    dh, dr = stored(g.standard_normal((rows, F)), it), stored(g.standard_normal((rows, F)), rt)
    args = (dev(r, rt), dev(o, it), dev(wp), dev(wq), dev(gate))
    rn, h = cuda_lib.block_norm_fwd(*args, scale=scale)
    rr, hr = lo.block_norm_fwd(r, o, wp, wq, gate, scale)
    close("residual", rn, rr)
    close("h", h, hr)
    for up in (dr, None):
        ref = lo.block_norm_bwd(r, o, wp, wq, gate, dh, up, scale)
        got = cuda_lib.block_norm_bwd(*args, dev(dh, it), dev(up, rt), scale=scale)
        assert set(got) == set(ref)
        for k, v in got.items():
            close(k, v, ref[k])


@pytest.mark.parametrize("rows,F,shift", [(300, 1028, 0), (40, 512, 4), (40, 520, 4), (40, 512, 1)])
def test_block_norm_bf16_rows_of_less_alignment(cuda_lib, rows, F, shift):
    """bf16 layer and residual whose width or address admits only shorter accesses."""
    import torch
    it, g = torch.bfloat16, np.random.default_rng(rows + F + shift)
    r, o, dh, dr = (stored(g.standard_normal((rows, F)), it) for _ in range(4))
    wp, wq = (stored(1 + 0.1 * g.standard_normal(F), torch.float32) for _ in range(2))

    def at(v):
        buf = torch.empty(rows * F + shift, dtype=it, device="cuda")[shift:].view(rows, F)
        return buf.copy_(dev(v, it))

    rn, h = cuda_lib.block_norm_fwd(at(r), at(o), dev(wp), dev(wq))
    rr, hr = lo.block_norm_fwd(r, o, wp, wq, None, 1.0)
    close("residual", rn, rr)
    close("h", h, hr)
    ref = lo.block_norm_bwd(r, o, wp, wq, None, dh, dr, 1.0)
    got = cuda_lib.block_norm_bwd(at(r), at(o), dev(wp), dev(wq), None, at(dh), at(dr))
    for k, v in got.items():
        close(k, v, ref[k])


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,F", [(700, 1030), (2, 2), (5, 8190)])
def test_block_norm_even_widths(cuda_lib, io, res, rows, F):
    gates = 2 if rows % 2 == 0 else 5
    test_block_norm_matches_oracle(cuda_lib, (rows, F, io, res, True, gates, 0.5))


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_block_norm_every_block_size(cuda_lib, io, res):
    """Widths that fill blocks of 32 to 512 threads, one column fewer, and narrower rows:
    every size of the rows' ring in shared memory."""
    for nt in range(32, 513, 32):
        for F in (16 * nt, 16 * nt - 1, 16 * nt - 248):
            test_block_norm_matches_oracle(cuda_lib, (3, F, io, res, True, 3, 0.5))

@pytest.mark.parametrize("rows,F,gates,io,post", [
    (70000, 5, 70000, "bf16", True),     # a gate row per row, more than a grid has block rows
    (140000, 8, 70000, "f32", False),    # two rows a gate row
    (65534, 4, 65534, "bf16", True),     # the first count past what one grid covers
    (65533, 4, 65533, "bf16", True)])
def test_block_norm_many_gate_rows(cuda_lib, rows, F, gates, io, post):
    test_block_norm_matches_oracle(cuda_lib, (rows, F, io, "f32", post, gates, 0.5))


def test_block_norm_in_place_and_unaligned_rows(cuda_lib):
    import torch
    r = torch.randn(33, 64, device="cuda")
    o = torch.randn(33, 64, device="cuda").to(torch.bfloat16)
    w = torch.rand(64, device="cuda")
    rn, h = cuda_lib.block_norm_fwd(r, o, w, w)
    # the same numbers at an address that is only element-aligned
    buf = torch.empty(33 * 64 + 1, device="cuda")[1:].view(33, 64).copy_(r)
    ob = torch.empty(33 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(33, 64).copy_(o)
    rn2, h2 = cuda_lib.block_norm_fwd(buf, ob, w, w)
    assert torch.allclose(rn, rn2, rtol=1e-6, atol=1e-6)
    assert torch.allclose(h.float(), h2.float(), rtol=2 ** -7, atol=1e-5)
    a, b = cuda_lib.block_norm_fwd(r, o, w, w, residual_out=r, h=o)
    assert a is r and b is o and torch.equal(r, rn) and torch.equal(o, h)


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,F", [(1000, 1001), (500, 3001), (500, 8191), (700, 2048), (500, 4100)])
def test_block_norm_in_place(cuda_lib, rows, F, io, res):
    """Several rows a block, in every way that rows are read: 4, 8 and 16 single columns
    a thread, whole pieces, and pieces with a remainder.  The bits of the call with
    outputs of its own."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows + F)
    r, o = (torch.randn(rows, F, generator=g, device="cuda").to(types(t)[0]) for t in (res, io))
    w, v = (torch.rand(F, generator=g, device="cuda") + 0.5 for _ in range(2))
    gate = torch.randn(5, F, generator=g, device="cuda")
    want = cuda_lib.block_norm_fwd(r, o, w, v, gate, scale=0.5)
    got = cuda_lib.block_norm_fwd(r, o, w, v, gate, scale=0.5, residual_out=r, h=o)
    assert got[0] is r and got[1] is o
    assert torch.equal(r, want[0]) and torch.equal(o, want[1])


def test_block_norm_zero_rows(cuda_lib):
    import torch
    r, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    rn, h = cuda_lib.block_norm_fwd(r, r, w)
    assert rn.shape == h.shape == (0, 64)
    got = cuda_lib.block_norm_bwd(r, r, w, w, None, r)
    assert torch.count_nonzero(got["dw_pre"]) == 0 and torch.count_nonzero(got["dw_post"]) == 0


# --------------------------------------------------------------------- refusals

def test_refusals(cuda_lib):
    import torch
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    x, w = z(2, 5, 8), z(8, 4)
    for bad in (dict(w=z(8, 5)), dict(w=z(8, 1))):      # windows outside 2 .. 4
        with pytest.raises(cuda_lib.SSDError) as e:
            cuda_lib.causal_conv_fwd(x, bad["w"])
        assert e.value.status == 2
    with pytest.raises(ValueError):
        cuda_lib.causal_conv_fwd(x, z(7, 4))
    with pytest.raises(ValueError):
        cuda_lib.causal_conv_fwd(x.transpose(1, 2), z(5, 4))          # channels not contiguous
    with pytest.raises(ValueError):
        cuda_lib.causal_conv_fwd(x.cpu(), w.cpu())
    with pytest.raises(TypeError):
        cuda_lib.causal_conv_fwd(x.half(), w)
    with pytest.raises(TypeError):
        cuda_lib.causal_conv_fwd(x, w, lengths=z(2, d=torch.int64))
    with pytest.raises(cuda_lib.SSDError):
        cuda_lib.causal_conv_fwd(x, w, out_dtype=torch.bfloat16)      # f32 in, bf16 out
    with pytest.raises(cuda_lib.SSDError):                            # more rows than states
        cuda_lib.causal_conv_step(x[:, 0], z(1, 3, 8), w)
    A, B = z(8, 16), z(2, 5, 1, 16)
    with pytest.raises(ValueError):
        cuda_lib.selective_scan_fwd(x, z(2, 4, 8), None, A, B, B)
    with pytest.raises(cuda_lib.SSDError) as e:
        cuda_lib.selective_scan_fwd(x, x, None, z(8, 65), z(2, 5, 1, 65), z(2, 5, 1, 65))
    assert e.value.status == 2
    with pytest.raises(cuda_lib.SSDError) as e:
        cuda_lib.selective_scan_fwd(x, x, None, A, z(2, 5, 3, 16), z(2, 5, 3, 16))
    assert e.value.status == 1                                        # 8 channels in 3 groups
    with pytest.raises(ValueError):
        cuda_lib.selective_scan_fwd(x, x, None, A, B, B, workspace=z(0, d=torch.uint8))
    with pytest.raises(ValueError):
        cuda_lib.ssd_step(z(2, 4, 8), z(2, 4), None, z(4), z(2, 1, 16), z(2, 1, 16), z(2, 4, 8, 8))
    r, f = z(6, 8), z(8)
    with pytest.raises(ValueError):
        cuda_lib.block_norm_fwd(r, r, f, gate=z(4, 8))                # 4 gate rows, 6 rows
    with pytest.raises(cuda_lib.SSDError) as e:
        cuda_lib.block_norm_fwd(z(1, 8193), z(1, 8193), z(8193))
    assert e.value.status == 2
    with pytest.raises(cuda_lib.SSDError) as e:                       # bf16 residual, f32 layer
        cuda_lib.block_norm_fwd(r.bfloat16(), r, f)
    assert e.value.status == 2


# ------------------------------------------------- tensors of more than 2^31 elements

def test_step_of_a_cache_past_32_bits(cuda_lib):
    """70000 slots of 4 x 64 x 128 states: the last slot's offset is past 2^31."""
    import torch
    g = np.random.default_rng(1)
    state = torch.empty(70000, 4, 64, 128, device="cuda")
    slots = dev(np.array([3, 69999]), torch.int32)
    state[3] = state[69999] = dev(g.standard_normal((4, 64, 128)))
    before = state[3].clone()

    def twice(*shape):
        t = dev(g.standard_normal((1,) + shape), torch.bfloat16)
        return t.expand(2, *shape).contiguous()

    y = cuda_lib.ssd_step(twice(4, 64), twice(4), None, dev(-np.ones(4)), twice(1, 128),
                          twice(1, 128), state, slots=slots)
    assert torch.equal(y[0], y[1]) and torch.equal(state[3], state[69999])
    assert not torch.equal(state[3], before)


def test_conv_past_32_bits(cuda_lib):
    """The last positions of 1.2 M x 1792 inputs, against a call on them alone."""
    import torch
    T, C, tail = 1200000, 1792, 67
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(1, T, C, generator=gen, device="cuda", dtype=torch.bfloat16)
             for _ in range(2))
    w = torch.randn(C, 4, generator=gen, device="cuda")
    xt, dt = x[:, -tail:], dy[:, -tail:]
    y, _ = cuda_lib.causal_conv_fwd(x, w)
    yt, _ = cuda_lib.causal_conv_fwd(xt, w)
    assert torch.equal(y[:, 3 - tail:], yt[:, 3:])
    del y
    dx = cuda_lib.causal_conv_bwd(x, w, None, dy)["dx"]
    dxt = cuda_lib.causal_conv_bwd(xt, w, None, dt)["dx"]
    assert torch.equal(dx[:, 3 - tail:], dxt[:, 3:])


def test_scan_past_32_bits(cuda_lib):
    """The last positions of 1.15 M x 1920 inputs, against a call that goes on from the
    state before them.  Both round to bf16, from ranges cut at other places."""
    import torch
    T, D, N, tail = 1150000, 1920, 4, 96
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    x, dt, dout = rand(1, T, D), rand(1, T, D), rand(1, T, D)
    B, C = rand(1, T, 1, N), rand(1, T, 1, N)
    A, bias = -torch.rand(D, N, generator=gen, device="cuda") - 0.1, torch.full((D,), -3.0, device="cuda")
    head, rest = T - tail, slice(T - tail, None)
    _, state = cuda_lib.selective_scan_fwd(x[:, :head], dt[:, :head], bias, A, B[:, :head], C[:, :head])
    part = (x[:, rest], dt[:, rest], bias, A, B[:, rest], C[:, rest])

    def same(a, b):
        a, b = a.double(), b.double()
        assert bool(torch.isfinite(a).all()) and (a - b).norm() <= 2.0 ** -8 * b.norm()

    out, fin = cuda_lib.selective_scan_fwd(x, dt, bias, A, B, C)
    want, wfin = cuda_lib.selective_scan_fwd(*part, init_states=state)
    same(out[:, rest], want)
    same(fin, wfin)
    del out
    got = cuda_lib.selective_scan_bwd(x, dt, bias, A, B, C, None, None, dout)
    want = cuda_lib.selective_scan_bwd(*part, None, None, dout[:, rest], init_states=state)
    for k in ("dx", "ddt", "dB", "dC"):
        same(got[k][:, rest], want[k])


def test_block_norm_past_32_bits(cuda_lib):
    """The last rows of 540000 x 4096, against a call on them alone (rows are independent)."""
    import torch
    rows, F, tail = 540000, 4096, 5
    gen = torch.Generator(device="cuda").manual_seed(4)
    r, o, dh = (torch.randn(rows, F, generator=gen, device="cuda", dtype=torch.bfloat16)
                for _ in range(3))
    w, v = (torch.rand(F, generator=gen, device="cuda") + 0.5 for _ in range(2))
    rn, h = cuda_lib.block_norm_fwd(r, o, w, v)
    rt, ht = cuda_lib.block_norm_fwd(r[-tail:], o[-tail:], w, v)
    assert torch.equal(rn[-tail:], rt) and torch.equal(h[-tail:], ht)
    del rn, h
    got = cuda_lib.block_norm_bwd(r, o, w, v, None, dh)
    want = cuda_lib.block_norm_bwd(r[-tail:], o[-tail:], w, v, None, dh[-tail:])
    assert all(torch.equal(got[k][-tail:], want[k]) for k in ("dresidual", "do"))


@pytest.mark.parametrize("T,D,dtype", [(3000000, 17, "bf16"), (64 * 65535 * 32, 1, "f32")])
def test_scan_of_the_longest_sequences(cuda_lib, T, D, dtype):
    """As test_scan_past_32_bits, at lengths up to the backward's limit."""
    import torch
    it, N, tail = types(dtype)[0], 2, 96
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=it)

    x, dt, dout = rand(1, T, D), rand(1, T, D), rand(1, T, D)
    B, C = rand(1, T, 1, N), rand(1, T, 1, N)
    A, bias = -torch.rand(D, N, generator=gen, device="cuda") - 0.1, torch.full((D,), -3.0, device="cuda")
    cut = lambda s: (x[:, s], dt[:, s], bias, A, B[:, s], C[:, s])  # noqa: E731
    _, state = cuda_lib.selective_scan_fwd(*cut(slice(0, T - tail)))
    rest = slice(T - tail, T)

    def same(a, b):
        a, b = a.double(), b.double()
        assert bool(torch.isfinite(a).all()) and (a - b).norm() <= 2.0 ** -8 * b.norm()

    out, fin = cuda_lib.selective_scan_fwd(x, dt, bias, A, B, C)
    want, wfin = cuda_lib.selective_scan_fwd(*cut(rest), init_states=state)
    same(out[:, rest], want)
    same(fin, wfin)
    got = cuda_lib.selective_scan_bwd(x, dt, bias, A, B, C, None, None, dout)
    want = cuda_lib.selective_scan_bwd(*cut(rest), None, None, dout[:, rest], init_states=state)
    for k in ("dx", "ddt", "dB", "dC"):
        same(got[k][:, rest], want[k])
