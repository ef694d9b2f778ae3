"""The norm of queries and keys at frequencies where its rotation can go wrong, against
the fp64 oracle (``oracle/delta_ops.py``) on a GPU."""
import numpy as np
import pytest

from oracle import delta_ops as do
from test_delta_ops import close, dev

pytestmark = pytest.mark.gpu


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
