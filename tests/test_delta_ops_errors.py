"""Argument checks of the gated delta rule's and the query / key norm's entry points:
every status below is returned, and every exception raised, before anything is launched, so
no GPU is needed."""
import ctypes

import pytest
import torch

import state_space_model_sm_gb300 as ssd
from state_space_model_sm_gb300 import _native, layer_ops
from test_current_device import CountingLibrary, t

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
D = ctypes.c_void_p(256)  # an aligned stand-in address, never dereferenced
ODD = ctypes.c_void_p(257)
BIG = ctypes.c_size_t(1 << 46)


@pytest.fixture(scope="module")
def lib():
    ssd.build()
    return ssd.load_library()


def delta(**kw):
    a = dict(batch=2, seqlen=16, nheads=4, headdim=8, dstate=16, ngroups=2, q_row_stride=0, k_row_stride=0,
             v_row_stride=0, q_batch_stride=0, k_batch_stride=0, v_batch_stride=0, scale=1.0, in_dtype=1,
             out_dtype=1)
    a.update(kw)
    return _native.DeltaShape(*a.values())


def qk(**kw):
    a = dict(batch=2, seqlen=16, q_heads=4, k_heads=2, headdim=16, rotary=8, q_row_stride=0, k_row_stride=0,
             q_batch_stride=0, k_batch_stride=0, eps=1e-6, l2=0, interleaved=0, in_dtype=1, out_dtype=1)
    a.update(kw)
    return _native.QkNormShape(*a.values())


def fwd(lib, s, a=None, ws=D, n=BIG):
    a = a or [D, D, D, D, None, D, D, None, None, D, None]
    return lib.ssd_gated_delta_fwd(s, *a, ws, n, None)


def bwd(lib, s, a=None, ws=D, n=BIG):
    a = a or [D, D, D, D, None, D, D, None, None, D, None, D, D, D, D, D, None, None, None]
    return lib.ssd_gated_delta_bwd(s, *a, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(nheads=0), INVALID),
    (dict(headdim=0), INVALID), (dict(dstate=0), INVALID), (dict(ngroups=0), INVALID),
    (dict(ngroups=3), INVALID), (dict(in_dtype=3), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(in_dtype=0, out_dtype=1), UNSUPPORTED), (dict(dstate=129), UNSUPPORTED),
    (dict(headdim=257), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(nheads=65536), UNSUPPORTED), (dict(seqlen=1 << 30), UNSUPPORTED),
    (dict(batch=60000, nheads=60000), UNSUPPORTED), (dict(q_row_stride=31), INVALID),
    (dict(k_row_stride=31), INVALID), (dict(v_row_stride=31), INVALID),
    (dict(q_row_stride=32, q_batch_stride=-1), INVALID)])
def test_delta_shapes(lib, kw, code):
    s = delta(**kw)
    assert fwd(lib, s) == code and bwd(lib, s) == code
    assert lib.ssd_gated_delta_fwd_workspace_size(s) == 0
    assert lib.ssd_gated_delta_bwd_workspace_size(s) == 0


def test_delta_pointers_and_workspace(lib):
    s = delta()
    a = [D, D, D, D, None, D, D, None, None, D, None]
    for i in (0, 1, 2, 3, 5, 6, 9):
        for bad in (None, ODD):
            assert fwd(lib, s, a[:i] + [bad] + a[i + 1:]) == INVALID
    for i in (4, 7, 8, 10):
        assert fwd(lib, s, a[:i] + [ODD] + a[i + 1:]) == INVALID
    need = lib.ssd_gated_delta_fwd_workspace_size(s)
    assert need > 0
    for ws, n in ((None, BIG), (ODD, BIG), (D, ctypes.c_size_t(need - 1))):
        assert fwd(lib, s, ws=ws, n=n) == WORKSPACE
    b = [D, D, D, D, None, D, D, None, None, D, None, D, D, D, D, D, None, None, None]
    for i in (0, 1, 2, 3, 5, 6, 9, 11, 12, 13, 14, 15):
        for bad in (None, ODD):
            assert bwd(lib, s, b[:i] + [bad] + b[i + 1:]) == INVALID
    for i in (4, 7, 8, 10, 16, 17, 18):
        assert bwd(lib, s, b[:i] + [ODD] + b[i + 1:]) == INVALID
    more = lib.ssd_gated_delta_bwd_workspace_size(s)
    assert more > need
    for ws, n in ((None, BIG), (ODD, BIG), (D, ctypes.c_size_t(more - 1))):
        assert bwd(lib, s, ws=ws, n=n) == WORKSPACE
    assert fwd(lib, None) == INVALID and bwd(lib, None) == INVALID


def test_delta_workspace_grows_with_the_sequence(lib):
    sizes = [lib.ssd_gated_delta_bwd_workspace_size(delta(seqlen=n)) for n in (64, 65, 128, 1 << 20)]
    # chunks of 64 tokens, and the head blocks' parts of dq and dk token by token
    assert sizes[0] < sizes[1] < sizes[2] < sizes[3]


@pytest.mark.parametrize("kw,code", [
    (dict(seqlen=2), INVALID), (dict(batch=0), INVALID), (dict(ngroups=3), INVALID),
    (dict(dstate=257), UNSUPPORTED), (dict(headdim=1 << 14), UNSUPPORTED),
    (dict(batch=1 << 24), UNSUPPORTED), (dict(in_dtype=0, out_dtype=1), UNSUPPORTED),
    (dict(v_row_stride=31), INVALID)])
def test_step_shapes(lib, kw, code):
    s = delta(**{"seqlen": 1, **kw})
    assert lib.ssd_gated_delta_step(s, D, D, D, D, None, D, D, D, D, 8, D, None) == code


def test_step_pointers(lib):
    s = delta(seqlen=1)
    a = [D, D, D, D, None, D, D, D, None]
    for i in (0, 1, 2, 3, 5, 6, 7):
        for bad in (None, ODD):
            assert lib.ssd_gated_delta_step(s, *(a[:i] + [bad] + a[i + 1:]), 8, D, None) == INVALID
    for i in (4, 8):
        assert lib.ssd_gated_delta_step(s, *(a[:i] + [ODD] + a[i + 1:]), 8, D, None) == INVALID
    for y in (None, ODD):
        assert lib.ssd_gated_delta_step(s, *a, 8, y, None) == INVALID
    assert lib.ssd_gated_delta_step(s, *a, 0, D, None) == INVALID
    assert lib.ssd_gated_delta_step(s, *a, 1, D, None) == INVALID  # two rows, one slot, no list


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(q_heads=0), INVALID),
    (dict(k_heads=0), INVALID), (dict(headdim=0), INVALID), (dict(rotary=-2), INVALID),
    (dict(rotary=7), INVALID), (dict(rotary=18), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(in_dtype=2), INVALID),
    (dict(in_dtype=0, out_dtype=1), UNSUPPORTED), (dict(headdim=1025), UNSUPPORTED),
    (dict(q_heads=65536), UNSUPPORTED), (dict(batch=1 << 20, seqlen=1 << 20), UNSUPPORTED),
    (dict(q_row_stride=63), INVALID), (dict(k_row_stride=31), INVALID),
    (dict(k_row_stride=32, k_batch_stride=-5), INVALID)])
def test_qk_shapes(lib, kw, code):
    s = qk(**kw)
    assert lib.ssd_qk_norm_fwd(s, D, D, None, None, D, None, D, D, None) == code
    assert lib.ssd_qk_norm_bwd(s, D, D, None, None, D, None, D, D, D, D, None, None, D, BIG, None) == code
    assert lib.ssd_qk_norm_workspace_size(s) == 0


def test_qk_pointers(lib):
    s = qk()
    a = [D, D, None, None, D, None, D, D]
    for i in (0, 1, 4, 6, 7):
        for bad in (None, ODD):
            assert lib.ssd_qk_norm_fwd(s, *(a[:i] + [bad] + a[i + 1:]), None) == INVALID
    for i in (2, 3, 5):
        assert lib.ssd_qk_norm_fwd(s, *(a[:i] + [ODD] + a[i + 1:]), None) == INVALID
    b = [D, D, D, D, D, None, D, D, D, D, D, D]
    for i in (0, 1, 4, 6, 7, 8, 9):
        for bad in (None, ODD):
            assert lib.ssd_qk_norm_bwd(s, *(b[:i] + [bad] + b[i + 1:]), D, BIG, None) == INVALID
    for i in (2, 3, 10, 11):  # weights and their gradients go together
        assert lib.ssd_qk_norm_bwd(s, *(b[:i] + [None] + b[i + 1:]), D, BIG, None) == INVALID
    need = lib.ssd_qk_norm_workspace_size(s)
    for ws, n in ((None, BIG), (ODD, BIG), (D, ctypes.c_size_t(need - 1))):
        assert lib.ssd_qk_norm_bwd(s, *b, ws, n, None) == WORKSPACE


# ------------------------------------------------------------- the bindings

def calls():
    q, v, g, h = t(2, 5, 2, 16), t(2, 5, 4, 8), t(2, 5, 4), t(4)
    q1, v1, g1, st = t(2, 2, 16), t(2, 4, 8), t(2, 4), t(3, 4, 8, 16)
    slots = t(2, dtype=torch.int32)
    pos, freq = t(2, 5, dtype=torch.int32), t(4)
    return {
        "gated_delta_fwd": lambda **k: ssd.gated_delta_fwd(**{**dict(
            q=q, k=q, v=v, dt=g, dt_bias=h, A=h, beta=g), **k}),
        "gated_delta_bwd": lambda **k: ssd.gated_delta_bwd(**{**dict(
            q=q, k=q, v=v, dt=g, dt_bias=h, A=h, beta=g, dy=v), **k}),
        "gated_delta_step": lambda **k: ssd.gated_delta_step(**{**dict(
            q=q1, k=q1, v=v1, dt=g1, dt_bias=h, A=h, beta=g1, state=st, slots=slots), **k}),
        "gated_delta_step, checked one by one": lambda **k: ssd.gated_delta_step(**{**dict(
            q=q1, k=q1, v=v1, dt=g1, dt_bias=h, A=h, beta=g1, state=st, slots=slots,
            out_dtype=torch.float32), **k}),
        "qk_norm_fwd": lambda **k: ssd.qk_norm_fwd(**{**dict(
            q=q, k=q, w_q=t(16), w_k=t(16), freq=freq, positions=pos), **k}),
        "qk_norm_bwd": lambda **k: ssd.qk_norm_bwd(**{**dict(
            q=q, k=q, w_q=t(16), w_k=t(16), freq=freq, positions=pos, dq_out=q, dk_out=q), **k}),
    }


@pytest.fixture
def placed(monkeypatch):
    """A machine whose current device is cuda:1, where the tensors say they live."""
    from state_space_model_sm_gb300 import delta_ops
    lib = CountingLibrary()
    for m in (layer_ops, delta_ops):
        monkeypatch.setattr(m, "_current_device", lambda: 1)
        monkeypatch.setattr(m, "_native_lib", lambda: lib)
        monkeypatch.setattr(m, "_stream", lambda dev: 0)
    return lib


@pytest.mark.parametrize("name", list(calls()))
def test_tensors_of_another_device_are_refused(placed, monkeypatch, name):
    from state_space_model_sm_gb300 import delta_ops
    for m in (layer_ops, delta_ops):
        monkeypatch.setattr(m, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1, but the current device is cuda:0"):
        calls()[name]()
    assert placed.calls == []


WRONG = {
    "gated_delta_fwd": [
        dict(q=t(2, 5, 16)), dict(q=t(2, 6, 2, 16)), dict(k=t(2, 5, 2, 8)), dict(k=t(2, 5, 2, 16, dtype=torch.bfloat16)),
        dict(v=t(2, 5, 8)), dict(dt=t(2, 5)), dict(beta=t(2, 4, 5)), dict(A=t(5)), dict(dt_bias=t(3)),
        dict(A=t(4, dtype=torch.float64)), dict(init_states=t(2, 4, 16, 8)), dict(lengths=t(2)),
        dict(lengths=t(3, dtype=torch.int32)), dict(out_dtype=torch.float16), dict(y=t(2, 5, 4, 9)),
        dict(final_states=t(2, 4, 8, 16, dtype=torch.bfloat16)), dict(v=t(2, 5, 8, 4).transpose(2, 3)),
        dict(workspace=t(1, dtype=torch.uint8))],
    "gated_delta_bwd": [
        dict(dy=t(2, 5, 4, 7)), dict(dy=t(2, 5, 4, 8, dtype=torch.bfloat16)), dict(dfinal_states=t(2, 4, 8, 8)),
        dict(out=dict(dq=t(2, 5, 2, 15))), dict(out=dict(dA=t(4, dtype=torch.bfloat16)))],
    "gated_delta_step": [
        dict(state=t(3, 4, 8, 8)), dict(state=t(3, 4, 8)), dict(state=t(3, 4, 8, 16, dtype=torch.bfloat16)),
        dict(slots=t(2)), dict(slots=t(3, dtype=torch.int32)), dict(q=t(2, 16)), dict(k=t(2, 2, 8)),
        dict(dt=t(2, 2)), dict(y=t(2, 4, 9)), dict(state=t(3, 4, 16, 8).transpose(2, 3))],
    "qk_norm_fwd": [
        dict(q=t(5, 16)), dict(k=t(2, 2, 16)), dict(k=t(2, 5, 2, 8)), dict(w_q=t(8)), dict(w_k=t(16, 1)),
        dict(freq=t(9)), dict(freq=t(2, 2)), dict(freq=t(4, dtype=torch.float64)),
        dict(positions=t(2, dtype=torch.int32)), dict(positions=t(2, 5)),
        dict(q=t(2, 2, 16), k=t(2, 2, 16), positions=None), dict(q_out=t(2, 5, 2, 15)),
        dict(out_dtype=torch.float16)],
    "qk_norm_bwd": [
        dict(dq_out=t(2, 5, 2, 8)), dict(dk_out=t(2, 5, 2, 16, dtype=torch.bfloat16)), dict(out=dict(dw_q=t(8)))],
}


@pytest.mark.parametrize("name,kw", [(n, k) for n, v in WRONG.items() for k in v])
def test_wrong_arguments_raise_before_any_launch(placed, name, kw):
    with pytest.raises((ValueError, TypeError)):
        calls()[name](**kw)
    assert all(c.endswith("workspace_size") for c in placed.calls)


def test_tensors_of_the_cpu_are_refused():
    x, g, h = torch.zeros(1, 2, 1, 4), torch.zeros(1, 2, 1), torch.zeros(1)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.gated_delta_fwd(x, x, x, g, h, h, g)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.qk_norm_fwd(x, x)
