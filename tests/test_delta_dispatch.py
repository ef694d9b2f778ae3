"""The gated delta rule and the norm of queries and keys on both sides of their dispatch
rules: sizes at which a block takes several heads of a group, a warp several tokens, a lane
eight rows, and a sequence many segments, against the fp64 oracle on a GPU.  The rules are of
152 SMs: 304 blocks for the gradients, 1216 for the outputs."""
import numpy as np
import pytest

import test_delta_ops as ops
from oracle import delta_ops as do
from test_delta_ops import close, dev, qk_case

pytestmark = pytest.mark.gpu


def ragged(B, T, seed=0):
    n = np.random.default_rng(seed).integers(0, T + 1, B)
    n[0], n[-1] = T, 0
    return n.tolist()


@pytest.mark.parametrize("case", [
    # B, T, H, G, P, N, dtype, init, lengths
    # one gradient block for the 2 heads of a group (320 blocks), two value tiles
    (160, 65, 2, 1, 72, 24, "bf16", True, ragged(160, 65)),
    (160, 65, 2, 1, 72, 24, "f32", True, ragged(160, 65)),
    (160, 65, 2, 1, 80, 100, "mixed", False, None),
    # two blocks for 3 heads in the outputs, one in the gradient (640 blocks)
    (320, 65, 3, 1, 24, 40, "bf16", False, ragged(320, 65, 1)),
    (320, 65, 3, 1, 24, 40, "f32", False, ragged(320, 65, 1)),
    # three blocks for 5 heads in the gradient (128 blocks)
    (64, 65, 5, 1, 40, 72, "bf16", True, ragged(64, 65, 2)),
    (64, 65, 5, 1, 40, 72, "f32", True, ragged(64, 65, 2)),
    # two groups, one block each in outputs and gradient (1280 blocks), three heads a group
    (80, 500, 6, 2, 16, 16, "bf16", True, ragged(80, 500, 3)),
    (80, 500, 6, 2, 16, 16, "f32", True, ragged(80, 500, 3)),
    # many heads that share their keys, whose gradients are summed in several blocks
    (160, 65, 64, 1, 8, 16, "mixed", True, None), (160, 65, 64, 1, 8, 16, "f32", False, None),
    (160, 65, 16, 1, 130, 16, "mixed", False, None), (160, 65, 64, 1, 8, 16, "bf16", False, None)])
def test_delta_of_several_heads_a_block(cuda_lib, case):
    ops.test_delta_matches_oracle(cuda_lib, case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_delta_of_one_head_in_many_segments(cuda_lib, dtype):
    """512 chunks in 32 segments, the longest that any rule makes, and a sequence that ends
    in the third of them."""
    ops.test_delta_matches_oracle(cuda_lib, (2, 32768, 1, 1, 8, 16, dtype, True, [32768, 3000]))


@pytest.mark.parametrize("case", [
    # (batch, seqlen), q heads, k heads, D, rotary, dtype, weights: a warp takes several tokens
    # (7296 warps forward, 2432 backward)
    ((2, 8000), 3, 2, 64, 64, "bf16", True), ((1, 9001), 2, 1, 32, 16, "f32", True),
    ((3, 3001), 2, 2, 20, 10, "mixed", True), ((2, 5000), 1, 3, 30, 30, "f32", False)])
@pytest.mark.parametrize("l2,interleaved", [(False, False), (True, True)])
def test_qk_norm_of_many_tokens(cuda_lib, case, l2, interleaved):
    """The weights' gradients are sums of independent terms over up to 48 thousand rows, each
    sum's roundings independent too: within the usual bounds."""
    import torch
    (B, T), HQ, HK, D, R, dtype, weights = case
    a, w, freq, gy, it, ot = qk_case((B, T), HQ, HK, D, R, dtype, weights)
    pos = np.tile(np.arange(T), (B, 1))
    kw = dict(l2=l2, interleaved=interleaved, eps=1e-5, out_dtype=ot)
    args = (dev(a["q"], it), dev(a["k"], it), dev(w[0]), dev(w[1]), dev(freq), None)
    out = cuda_lib.qk_norm_fwd(*args, **kw)
    got = cuda_lib.qk_norm_bwd(*args, dev(gy[0], it), dev(gy[1], it), **kw)
    for i, n in enumerate("qk"):
        rows = lambda m: m.reshape((B * T,) + m.shape[2:])  # noqa: E731
        ref = do.norm_fwd(rows(a[n]), w[i], freq, pos.ravel(), l2, interleaved, 1e-5)
        close(n + "_out", out[i], ref.reshape(a[n].shape))
        dx, dw = do.norm_bwd(rows(a[n]), w[i], freq, pos.ravel(), rows(gy[i]), l2, interleaved, 1e-5)
        close("d" + n, got["d" + n], dx.reshape(a[n].shape))
        if weights:
            close("dw_" + n, got["dw_" + n], dw)
    # a second call on another stream: the same bits
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = cuda_lib.qk_norm_bwd(*args, dev(gy[0], it), dev(gy[1], it), **kw)
    s.synchronize()
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("B,H,G,P,N,dtype", [
    # eight rows a lane: 8, 16 and 32 lanes a row
    (64, 64, 32, 64, 32, "bf16"), (65, 63, 21, 65, 20, "f32"), (64, 32, 8, 64, 64, "mixed"),
    (33, 63, 9, 65, 48, "bf16"), (17, 63, 63, 65, 100, "f32")])
def test_delta_step_of_many_rows(cuda_lib, B, H, G, P, N, dtype):
    ops.test_delta_step_matches_oracle(cuda_lib, B, H, G, P, N, dtype)


def test_norm_of_the_ssd_scans_inputs(cuda_lib):
    """The RMS form with rotation in front of the SSD scan: its B and C as keys and queries, from
    column ranges of one projection, against the two oracles in a row.  fp32: two parts' errors."""
    import torch
    a, w, freq, _, it, _ = qk_case((2, 128), 2, 2, 16, 8, "f32", True)
    g = np.random.default_rng(5)
    x, dt = g.standard_normal((2, 128, 4, 8)), g.standard_normal((2, 128, 4)) - 2
    A = -np.exp(0.3 * g.standard_normal(4))
    wide = torch.cat([dev(a["q"]).flatten(2), dev(a["k"]).flatten(2)], -1)
    c, b = (m.unflatten(-1, (2, 16)) for m in wide.split(32, -1))
    C, Bm = cuda_lib.qk_norm_fwd(c, b, dev(w[0]), dev(w[1]), dev(freq))
    x, dt, A = (m.astype(np.float32).astype(float) for m in (x, dt, A))  # as the kernels read them
    y, _ = cuda_lib.ssd_fwd(dev(x), dev(dt), None, dev(A), Bm, C, chunk_size=64)
    pos = np.tile(np.arange(128), 2)
    flat = lambda m: m.reshape((256,) + m.shape[2:])  # noqa: E731
    Cr, Br = (do.norm_fwd(flat(a[n]), w[i], freq, pos).reshape(a[n].shape) for i, n in enumerate("qk"))
    # the scan, token by token
    h, ref = np.zeros((2, 4, 8, 16)), np.zeros_like(x)
    delta = np.log1p(np.exp(dt))
    for t in range(128):
        bt, ct = np.repeat(Br[:, t], 2, 1), np.repeat(Cr[:, t], 2, 1)
        h = np.exp(delta[:, t] * A)[..., None, None] * h \
            + (delta[:, t, :, None] * x[:, t])[..., None] * bt[:, :, None]
        ref[:, t] = np.einsum("bhpn,bhn->bhp", h, ct)
    close("y", y, ref)
