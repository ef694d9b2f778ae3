"""The norm of queries and keys at frequencies where its rotation can go wrong, against
the fp64 oracle (``oracle/delta_ops.py``) on a GPU."""
import numpy as np
import pytest

from oracle import delta_ops as do
from test_delta_ops import close, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 2.0 ** 20, -2.0 ** 100])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 70])  # pieces of 16 bytes, single columns
def test_a_frequency_out_of_range_is_nan(cuda_lib, value, interleaved, D):
    """Its pair is NaN at every position but nothing else, forward and backward."""
    g = np.random.default_rng(D)
    x, dy = g.standard_normal((1, 5, 2, D)), g.standard_normal((1, 5, 2, D))
    freq, pairs = g.uniform(0.1, 1.0, D // 2), D // 2
    i = 3
    hit = np.zeros(D, bool)
    hit[[2 * i, 2 * i + 1] if interleaved else [i, i + pairs]] = True
    kw = dict(interleaved=interleaved, l2=True)
    want = cuda_lib.qk_norm_fwd(dev(x), dev(x), freq=dev(freq), **kw)[0].cpu().numpy()
    freq[i] = value
    got = cuda_lib.qk_norm_fwd(dev(x), dev(x), freq=dev(freq), **kw)[0].cpu().numpy()
    assert np.isnan(got[..., hit]).all() and np.array_equal(got[..., ~hit], want[..., ~hit])
    b = cuda_lib.qk_norm_bwd(dev(x), dev(x), None, None, dev(freq), None, dev(dy), dev(dy), **kw)
    assert bool(b["dq"].isnan().all())  # each value's gradient holds the row's sum


def test_the_largest_frequencies(cuda_lib):
    """Just under the limit and at the far positions: the fraction of a turn is what is left of
    2^51 radians.  The oracle's angle, a product of doubles, is good to 2^-53 of it, 2^-2
    radians at the far end, so it is formed from whole turns by integers here."""
    import torch
    from fractions import Fraction
    # 2 pi to 60 digits: 2^51 radians to 1e-44 of a turn
    two_pi = Fraction(2 * 314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    freq = np.array([2.0 ** 20 - 0.0625, 1234567.0 / 2, 3.0, 2.0 ** -40], np.float32)
    pos = np.array([(1 << 31) - 1, -(1 << 31), 12345, 0, -7])
    angle = np.array([[float((Fraction(float(f)) * int(p) / two_pi) % 1) * 2 * np.pi for f in freq] for p in pos])
    x = np.random.default_rng(1).standard_normal((5, 1, 8)).astype(np.float32)
    got = cuda_lib.qk_norm_fwd(dev(x), dev(x), freq=dev(freq),
                               positions=dev(pos, torch.int32))[0]
    n = do.norm_fwd(x)
    z = (n[..., :4] + 1j * n[..., 4:]) * np.exp(1j * angle)[:, None]
    close("q_out", got, np.concatenate([z.real, z.imag], -1))
