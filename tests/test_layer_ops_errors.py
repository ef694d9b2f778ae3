"""Argument checks of the layer operators' C entry points: every status below is
returned before anything is launched, so no GPU is needed."""
import ctypes

import pytest

import state_space_model_sm_gb300 as ssd
from state_space_model_sm_gb300 import _native

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
D = ctypes.c_void_p(256)  # an aligned stand-in address, never dereferenced
ODD = ctypes.c_void_p(257)
BIG = ctypes.c_size_t(1 << 40)


@pytest.fixture(scope="module")
def lib():
    ssd.build()
    return ssd.load_library()


def conv(**kw):
    a = dict(batch=2, seqlen=16, channels=8, width=4, x_row_stride=0, x_batch_stride=0, silu=1, in_dtype=1,
             out_dtype=1)
    a.update(kw)
    return _native.ConvShape(*a.values())


def sel(**kw):
    a = dict(batch=2, seqlen=16, channels=8, dstate=16, ngroups=1, z_row_stride=0, b_row_stride=0,
             c_row_stride=0, z_batch_stride=0, b_batch_stride=0, c_batch_stride=0, in_dtype=1, out_dtype=1)
    a.update(kw)
    return _native.SelectiveShape(*a.values())


def norm(**kw):
    a = dict(rows=8, features=64, ngates=0, eps=1e-5, scale=1.0, in_dtype=1, res_dtype=0)
    a.update(kw)
    return _native.BlockNormShape(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(channels=0), INVALID),
    (dict(width=0), INVALID), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED),
    (dict(in_dtype=3), INVALID), (dict(in_dtype=0, out_dtype=1), UNSUPPORTED),
    (dict(x_row_stride=7), INVALID), (dict(seqlen=1 << 30), UNSUPPORTED)])
def test_conv_shapes(lib, kw, code):
    s = conv(**kw)
    assert lib.ssd_causal_conv_fwd(s, D, D, None, None, None, D, None, None) == code
    assert lib.ssd_causal_conv_bwd(s, D, D, None, None, None, D, None, D, D, None, None, D, BIG,
                                   None) == code
    assert lib.ssd_causal_conv_step(s, D, D, D, None, None, 8, D, None) == code
    assert lib.ssd_causal_conv_workspace_size(s) == 0


def test_conv_pointers(lib):
    s = conv()
    for i in (0, 1, 5):
        a = [D, D, None, None, None, D, None]
        for bad in (None, ODD):
            a[i] = bad
            assert lib.ssd_causal_conv_fwd(s, *a, None) == INVALID
    a = [D, D, None, None, None, D, None, D, D, None, None]
    assert lib.ssd_causal_conv_bwd(s, *a, None, BIG, None) == WORKSPACE
    assert lib.ssd_causal_conv_bwd(s, *a, D, ctypes.c_size_t(4), None) == WORKSPACE
    for i in (0, 1, 5, 7, 8):
        b = list(a)
        b[i] = None
        assert lib.ssd_causal_conv_bwd(s, *b, D, BIG, None) == INVALID
    one = conv(seqlen=1)
    assert lib.ssd_causal_conv_step(s, D, D, D, None, None, 8, D, None) == INVALID  # seqlen 16
    assert lib.ssd_causal_conv_step(one, D, D, D, None, None, 1, D, None) == INVALID  # 2 rows
    assert lib.ssd_causal_conv_step(one, D, D, D, None, D, 0, D, None) == INVALID
    assert lib.ssd_causal_conv_step(one, D, None, D, None, D, 8, D, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(dstate=0), INVALID),
    (dict(ngroups=3), INVALID), (dict(dstate=65), UNSUPPORTED), (dict(in_dtype=2), INVALID),
    (dict(in_dtype=0, out_dtype=1), UNSUPPORTED), (dict(z_row_stride=7), INVALID),
    (dict(b_row_stride=15), INVALID), (dict(c_row_stride=1), INVALID),
    (dict(batch=65536), UNSUPPORTED)])
def test_scan_shapes(lib, kw, code):
    s = sel(**kw)
    assert lib.ssd_selective_scan_fwd(s, D, D, None, D, D, D, None, None, None, None, D, None, D,
                                      BIG, None) == code
    assert lib.ssd_selective_scan_bwd(s, D, D, None, D, D, D, None, None, None, None, D, None, D, D,
                                      D, D, D, None, None, None, None, D, BIG, None) == code
    assert lib.ssd_selective_scan_fwd_workspace_size(s) == 0
    assert lib.ssd_selective_scan_bwd_workspace_size(s) == 0


def test_scan_pointers(lib):
    s = sel()
    fwd = [D, D, None, D, D, D, None, None, None, None, D, None]
    for i in (0, 1, 3, 4, 5, 10):
        for bad in (None, ODD):
            a = list(fwd)
            a[i] = bad
            assert lib.ssd_selective_scan_fwd(s, *a, D, BIG, None) == INVALID, i
    assert lib.ssd_selective_scan_fwd(s, *fwd, None, BIG, None) == WORKSPACE
    bwd = [D, D, None, D, D, D, None, D, None, None, D, None, D, D, D, D, D, None, D, None, None]
    assert lib.ssd_selective_scan_bwd(s, *bwd, D, ctypes.c_size_t(64), None) == WORKSPACE
    for i in (0, 1, 3, 4, 5, 10, 12, 13, 14, 15, 16, 18):  # 18: dz, required with z
        a = list(bwd)
        a[i] = None
        assert lib.ssd_selective_scan_bwd(s, *a, D, BIG, None) == INVALID, i


def test_step_arguments(lib):
    one = sel(seqlen=1)
    a = [D, D, None, D, D, D, None, None, D, None]
    assert lib.ssd_selective_step(sel(), *a, 8, D, None) == INVALID       # seqlen 16
    assert lib.ssd_selective_step(one, *a, 1, D, None) == INVALID          # 2 rows, 1 state
    assert lib.ssd_selective_step(one, *a, 8, None, None) == INVALID
    assert lib.ssd_selective_step(sel(seqlen=1, dstate=257), *a, 8, D, None) == UNSUPPORTED
    s = ssd.make_shape(2, 1, 4, 64, 128, 1, 1, ssd.SSD_BF16, ssd.SSD_BF16)
    b = [D, D, None, D, D, D, None, D, None]
    assert lib.ssd_step(s, *b, 1, D, None) == INVALID
    assert lib.ssd_step(s, *b, 8, ODD, None) == INVALID
    for i in (0, 1, 3, 4, 5, 7):
        v = list(b)
        v[i] = None
        assert lib.ssd_step(s, *v, 8, D, None) == INVALID, i
    assert lib.ssd_step(ssd.make_shape(2, 1, 4, 64, 128, 3, 1), *b, 8, D, None) == INVALID
    assert lib.ssd_step(ssd.make_shape(2, 1, 4, 256, 128, 1, 1), *b, 8, D, None) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(features=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(ngates=3), INVALID), (dict(in_dtype=9), INVALID),
    (dict(features=8193), UNSUPPORTED), (dict(in_dtype=0, res_dtype=1), UNSUPPORTED)])
def test_block_norm_shapes(lib, kw, code):
    s = norm(**kw)
    g = D if kw.get("ngates") else None
    assert lib.ssd_block_norm_fwd(s, D, D, D, None, g, D, D, None) == code
    assert lib.ssd_block_norm_bwd(s, D, D, D, None, g, D, None, D, D, D, None, g, D, BIG,
                                  None) == code
    assert lib.ssd_block_norm_workspace_size(s) == 0


def test_block_norm_pointers(lib):
    s = norm()
    fwd = [D, D, D, None, None, D, D]
    for i in (0, 1, 2, 5, 6):
        a = list(fwd)
        a[i] = None
        assert lib.ssd_block_norm_fwd(s, *a, None) == INVALID
    assert lib.ssd_block_norm_fwd(s, D, D, D, None, D, D, D, None) == INVALID  # gate, ngates 0
    bwd = [D, D, D, None, None, D, None, D, D, D, None, None]
    assert lib.ssd_block_norm_bwd(s, *bwd, None, BIG, None) == WORKSPACE
    assert lib.ssd_block_norm_bwd(s, *bwd[:10], D, None, D, BIG, None) == INVALID  # dw_post alone
    assert lib.ssd_block_norm_fwd(norm(rows=0), *[None] * 7, None) == OK


def test_block_norm_row_limit(lib):
    """Too many rows is a limit, a gate that does not divide them a wrong argument."""
    for s, g, code in ((norm(rows=1 << 30), None, UNSUPPORTED),
                       (norm(rows=1 << 30, ngates=3), D, INVALID)):
        assert lib.ssd_block_norm_fwd(s, D, D, D, None, g, D, D, None) == code
        assert lib.ssd_block_norm_bwd(s, D, D, D, None, g, D, None, D, D, D, None, g, D, BIG,
                                      None) == code
        assert lib.ssd_block_norm_workspace_size(s) == 0
    assert lib.ssd_block_norm_workspace_size(norm(rows=(1 << 30) - 1)) > 0


@pytest.mark.parametrize("call", ["forward", "backward"])
def test_scan_stops_at_a_refused_launch(lib, call):
    """Without a GPU every launch is refused: the scan's first pass is the only one
    tried, since the others would read what it has not written."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the stand-in addresses must never reach a GPU")
    s = sel(seqlen=4096, dstate=64)  # several ranges; no pass needs more than 48 KB of shared memory
    before = lib.ssd_launch_count()
    if call == "forward":
        st = lib.ssd_selective_scan_fwd(s, D, D, None, D, D, D, None, None, None, None, D, None, D,
                                        BIG, None)
    else:
        st = lib.ssd_selective_scan_bwd(s, D, D, None, D, D, D, None, None, None, None, D, None, D,
                                        D, D, D, D, None, None, None, None, D, BIG, None)
    assert st == 4 and lib.ssd_launch_count() == before + 1  # SSD_ERR_CUDA


def test_scan_length_limits(lib):
    """The limits of the header, in the calls and in the size queries alike."""
    fwd = [D, D, None, D, D, D, None, None, None, None, D, None, None, BIG, None]
    bwd = [D, D, None, D, D, D, None, None, None, None, D, None, D, D, D, D, D, None, None, None,
           None, None, BIG, None]  # no workspace: nothing past the shape's check is launched
    top = 64 * 65535 * 32
    for kw, forward, backward in (
            (dict(batch=1, seqlen=top), WORKSPACE, WORKSPACE),
            (dict(batch=1, seqlen=top + 1), WORKSPACE, UNSUPPORTED),
            (dict(batch=1, seqlen=(1 << 30) - 1), WORKSPACE, UNSUPPORTED),
            (dict(batch=1, seqlen=1 << 30), UNSUPPORTED, UNSUPPORTED),
            (dict(batch=128, seqlen=1 << 24), WORKSPACE, WORKSPACE),      # batch * seqlen = 2^31
            (dict(batch=129, seqlen=1 << 24), WORKSPACE, UNSUPPORTED),
            (dict(batch=65, seqlen=1 << 24, ngroups=2), WORKSPACE, UNSUPPORTED),
            (dict(batch=65535, seqlen=1, channels=1 << 23, ngroups=1 << 23), UNSUPPORTED,
             UNSUPPORTED)):
        s = sel(**kw)
        assert lib.ssd_selective_scan_fwd(s, *fwd) == forward, kw
        assert lib.ssd_selective_scan_bwd(s, *bwd) == backward, kw
        assert (lib.ssd_selective_scan_fwd_workspace_size(s) == 0) == (forward == UNSUPPORTED), kw
        assert (lib.ssd_selective_scan_bwd_workspace_size(s) == 0) == (backward == UNSUPPORTED), kw


def test_conv_states_must_not_overlap(lib):
    """The final state is written before the initial one is used up, so going on in
    place would give wrong outputs: refused, at any overlap of the two."""
    s = conv(batch=2, width=4, channels=8)  # states of 2 x 3 x 8 bf16: 96 bytes
    at = ctypes.c_void_p
    for init, final in ((256, 256), (256, 350), (350, 256)):
        assert lib.ssd_causal_conv_fwd(s, D, D, None, at(init), None, D, at(final), None) == INVALID
