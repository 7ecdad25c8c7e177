"""The operators around the attention refuse bad arguments with the documented
status before anything reaches the GPU (CPU only): addresses here are made up and
never dereferenced."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import static_sparse_attention_b200 as ra
    return ra


MB = 1 << 20


def _rope(ra, **kw):
    a = dict(t=1 * MB, h=2 * MB, w=3 * MB, frames=10, grid_h=4, grid_w=5, t_pairs=22, h_pairs=21, w_pairs=21)
    a.update(kw)
    return ra.ra_rope(*(a[f] for f, _ in ra.ra_rope._fields_))


def _rows(ra, x, **kw):
    a = dict(x=x, stride_b=40 * 3 * 128, stride_n=3 * 128, stride_h=128, heads=1, weight_fp32=0, weight=9 * MB)
    a.update(kw)
    return ra.ra_head_rows(*(a[f] for f, _ in ra.ra_head_rows._fields_))


def _fwd(ra, q=None, k=None, q_out=20 * MB, k_out=21 * MB, B=2, n=40, d=128, rope=None, frame0=0, eps=1e-6):
    q = _rows(ra, 10 * MB) if q is None else q
    return ra.ra_qk_norm_rope(ctypes.byref(q) if q != 0 else None, ctypes.byref(k) if k is not None else None, q_out,
                              k_out, B, n, d, ctypes.byref(rope) if rope is not None else None, frame0, eps, None)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(q_out=None), dict(q_out=20 * MB + 8), dict(B=0), dict(B=70000), dict(n=-1), dict(eps=0.0),
    dict(eps=float("nan")), dict(eps=float("inf")),
])
def test_norm_rope_refuses(ra, kw):
    assert _fwd(ra, **kw) == ra.RA_ERR_INVALID_ARG
    assert ra.ra_last_error()


def test_norm_rope_refuses_what_is_too_large(ra):
    assert _fwd(ra, q=_rows(ra, 10 * MB, heads=60000, stride_h=0), B=60000, n=1000) == ra.RA_ERR_UNSUPPORTED
    assert _fwd(ra, q=_rows(ra, 10 * MB, stride_n=1 << 44)) == ra.RA_ERR_INVALID_ARG


def test_norm_rope_refuses_head_dims(ra):
    assert _fwd(ra, d=96) == ra.RA_ERR_UNSUPPORTED
    assert _fwd(ra, d=256) == ra.RA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=10 * MB + 2), dict(heads=0), dict(heads=65536), dict(weight=9 * MB + 4), dict(stride_n=3 * 128 + 4),
    dict(stride_b=-8), dict(weight=None),  # neither a norm nor a rotation
])
def test_norm_rope_refuses_rows(ra, kw):
    a = dict(x=10 * MB)
    a.update(kw)
    x = a.pop("x")
    assert _fwd(ra, q=_rows(ra, x, **a)) == ra.RA_ERR_INVALID_ARG
    assert _fwd(ra, k=_rows(ra, x, **a)) == ra.RA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,frame0", [
    (dict(t=None), 0), (dict(h=2 * MB + 4), 0), (dict(t_pairs=-1), 0), (dict(t_pairs=23), 0), (dict(t_pairs=65), 0),
    (dict(t_pairs=0, h_pairs=0, w_pairs=0), 0), (dict(frames=0), 0), (dict(grid_h=0), 0), (dict(grid_w=-3), 0),
    (dict(grid_h=1 << 16, grid_w=1 << 16), 0), (dict(), -1),
    (dict(), 9),               # 40 tokens are frames 9 and 10 of 10
    (dict(frames=1), 0),       # and two frames of 20 tokens
])
def test_norm_rope_refuses_tables(ra, kw, frame0):
    assert _fwd(ra, rope=_rope(ra, **kw), frame0=frame0) == ra.RA_ERR_INVALID_ARG
    assert ra.ra_last_error()


def test_norm_rope_refuses_aliases(ra):
    size = 2 * 40 * 128 * 2  # bytes of an output
    for out in (10 * MB, 10 * MB + 1024, 10 * MB - size + 16, 9 * MB - size + 16):
        assert _fwd(ra, q_out=out) == ra.RA_ERR_INVALID_ARG
        assert b"alias" in ra.ra_last_error()
    k = _rows(ra, 12 * MB)
    assert _fwd(ra, k=k, k_out=None) == ra.RA_ERR_INVALID_ARG
    assert _fwd(ra, k=k, q_out=20 * MB, k_out=20 * MB + size - 16) == ra.RA_ERR_INVALID_ARG
    assert _fwd(ra, k=k, q_out=12 * MB) == ra.RA_ERR_INVALID_ARG


def _bwd(ra, dx=20 * MB, dy=22 * MB, dw=24 * MB, ws=26 * MB, ws_bytes=None, strides=(40 * 128, 128, 128), k=None, dk=None,
         q=None, n=40, B=2, d=128):
    q = _rows(ra, 10 * MB) if q is None else q
    dq = ra.ra_head_grads(dy, dx, *strides, dw)
    need = ra.ra_qk_norm_rope_bwd_workspace_bytes(d) if ws_bytes is None else ws_bytes
    return ra.ra_qk_norm_rope_bwd(ctypes.byref(q), None if k is None else ctypes.byref(k), ctypes.byref(dq),
                                  None if dk is None else ctypes.byref(dk), B, n, d, None, 0, 1e-6, ws, need, None)


@pytest.mark.parametrize("kw", [
    dict(dx=None), dict(dy=None), dict(dx=20 * MB + 4), dict(dw=None), dict(dw=24 * MB + 2), dict(ws=None),
    dict(ws=26 * MB + 8), dict(ws_bytes=1000), dict(strides=(40 * 128, 128 + 2, 128)),
    dict(strides=(0, 128, 128)),           # batch elements on top of each other
    dict(strides=(40 * 128, 64, 128)),     # rows that overlap
    dict(strides=(39 * 128, 128, 128)),
    dict(dx=10 * MB), dict(dx=22 * MB + 64), dict(dw=10 * MB), dict(dw=20 * MB), dict(ws=22 * MB), dict(ws=24 * MB - 64),
    dict(dw=9 * MB), dict(ws=20 * MB + 32),
])
def test_norm_rope_bwd_refuses(ra, kw):
    assert _bwd(ra, **kw) == ra.RA_ERR_INVALID_ARG
    assert ra.ra_last_error()


def test_norm_rope_bwd_refuses_shared_gradients(ra):
    k = _rows(ra, 12 * MB, weight=9 * MB + 4096)
    for at in (20 * MB, 20 * MB + 128, 20 * MB + 128 * 2):  # the same rows, half a row on, a row on
        dk = ra.ra_head_grads(23 * MB, at, 40 * 128, 128, 128, 25 * MB)
        assert _bwd(ra, k=k, dk=dk) == ra.RA_ERR_INVALID_ARG
        assert b"alias" in ra.ra_last_error()
    dk = ra.ra_head_grads(23 * MB, 21 * MB, 40 * 128, 128, 128, 24 * MB)  # one gradient for both weights
    assert _bwd(ra, k=k, dk=dk) == ra.RA_ERR_INVALID_ARG
    assert _bwd(ra, k=k) == ra.RA_ERR_INVALID_ARG           # k without dk


def test_rope_table_refuses(ra):
    for args in ((None, 0, 4, 8, 1e4), (MB + 4, 0, 4, 8, 1e4), (MB, -1, 4, 8, 1e4), (MB, 0, 0, 8, 1e4), (MB, 0, 4, 0, 1e4),
                 (MB, 0, 4, 65, 1e4), (MB, (1 << 31) - 2, 4, 8, 1e4), (MB, 0, 4, 8, 1.0), (MB, 0, 4, 8, float("inf"))):
        assert ra.ra_rope_table(*args, None) == ra.RA_ERR_INVALID_ARG
        assert ra.ra_last_error()


def test_python_layer_refuses(ra):
    import torch
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        ra.qk_norm_rope(x, rope=None)  # not on a CUDA device
    with pytest.raises(ValueError):
        ra.rope3d(4, 4, 4, 64, axes=(3, 4, 4))
    with pytest.raises(ValueError):
        ra.rope3d(4, 4, 4, 64, axes=(32, 32, 2))
    assert ra.rope_axes(128) == (44, 42, 42) and sum(ra.rope_axes(64)) == 64


# ---------------------------------------------------------------- 8-bit key/value ring
def _append(ra, k=None, v=None, B=2, frames=2, d=128, s=20, W=4, frame=0, rope=None, eps=1e-6, k8=30 * MB, v8=31 * MB,
            ks=32 * MB, vs=33 * MB):
    k = _rows(ra, 10 * MB) if k is None else k
    v = _rows(ra, 12 * MB, weight=None) if v is None else v
    return ra.ra_cache8_append(ctypes.byref(k) if k != 0 else None, ctypes.byref(v), B, frames, d, s, W, frame,
                               None if rope is None else ctypes.byref(rope), eps, k8, v8, ks, vs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), 1), (dict(B=0), 1), (dict(d=80), 2), (dict(s=0), 1), (dict(W=0), 1), (dict(frames=0), 1),
    (dict(frames=5), 1),                        # two frames would share a slot
    (dict(frame=-1), 1), (dict(eps=0.0), 1), (dict(k8=None), 1), (dict(v8=31 * MB + 8), 1), (dict(ks=32 * MB + 2), 1),
    (dict(vs=None), 1), (dict(s=1 << 20, W=1 << 12), 2), (dict(k8=10 * MB), 1), (dict(v8=30 * MB + 64), 1),
    (dict(ks=12 * MB), 1), (dict(vs=32 * MB), 1), (dict(ks=9 * MB), 1),
])
def test_cache8_append_refuses(ra, kw, status):
    assert _append(ra, **kw) == status
    assert ra.ra_last_error()


def test_cache8_append_refuses_rows_and_ropes(ra):
    assert _append(ra, v=_rows(ra, 12 * MB)) == ra.RA_ERR_INVALID_ARG                       # v with a weight
    assert _append(ra, v=_rows(ra, 12 * MB, weight=None, heads=2)) == ra.RA_ERR_INVALID_ARG  # other heads than k
    assert _append(ra, k=_rows(ra, 10 * MB + 8)) == ra.RA_ERR_INVALID_ARG
    assert _append(ra, rope=_rope(ra, grid_h=3)) == ra.RA_ERR_INVALID_ARG                   # 15 tokens, not 20
    assert _append(ra, rope=_rope(ra), frame=9) == ra.RA_ERR_INVALID_ARG                    # frames 9 and 10 of 10
    assert _append(ra, rope=_rope(ra), frame=1 << 40) == ra.RA_ERR_INVALID_ARG


def _attend(ra, Q=10 * MB, k8=30 * MB, v8=31 * MB, ks=32 * MB, vs=33 * MB, O=40 * MB, B=2, H=1, d=128, nq=3, s=20, W=4,
            held=3, counts=None, scale=0.1, lse=None, ws=50 * MB, ws_bytes=None):
    need = ctypes.c_size_t()
    st = ra.ra_cache8_attention_workspace_bytes(B, H, d, nq, s, W, held, ctypes.byref(need))
    got = ra.ra_cache8_attention(Q, k8, v8, ks, vs, O, B, H, d, nq, s, W, held, counts, scale, lse, ws,
                                 need.value if ws_bytes is None else ws_bytes, None)
    assert st == ra.RA_OK or got == st
    return got


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), 1), (dict(O=None), 1), (dict(Q=10 * MB + 8), 1), (dict(k8=None), 1), (dict(B=0), 1), (dict(H=70000), 1),
    (dict(d=32), 2), (dict(nq=0), 1), (dict(nq=1 << 25), 1), (dict(held=5), 1), (dict(held=-1), 1), (dict(s=0), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(counts=60 * MB + 2), 1), (dict(lse=61 * MB + 1), 1),
    (dict(O=10 * MB), 1), (dict(O=30 * MB), 1), (dict(lse=32 * MB), 1), (dict(lse=40 * MB), 1), (dict(counts=40 * MB), 1),
    (dict(s=1 << 20, W=1 << 12), 2), (dict(s=1 << 20, W=1 << 10, H=60000, B=60000), 2),
    (dict(H=60000, B=60000, nq=1000), 2),
])
def test_cache8_attention_refuses(ra, kw, status):
    assert _attend(ra, **kw) == status
    assert ra.ra_last_error()


def test_cache8_attention_refuses_workspaces(ra):
    long = dict(s=1, W=20000, held=20000, k8=130 * MB, v8=140 * MB, ks=150 * MB, vs=151 * MB)
    need = ctypes.c_size_t()
    assert ra.ra_cache8_attention_workspace_bytes(2, 1, 128, 3, 1, 20000, 20000, ctypes.byref(need)) == ra.RA_OK
    assert need.value > 0
    for kw in (dict(ws=None), dict(ws_bytes=need.value - 1), dict(ws=50 * MB + 8), dict(ws=40 * MB), dict(ws=130 * MB)):
        assert _attend(ra, **long, **kw) == ra.RA_ERR_INVALID_ARG
        assert ra.ra_last_error()
    assert ra.ra_cache8_attention_workspace_bytes(2, 1, 128, 3, 20, 4, 3, None) == ra.RA_ERR_INVALID_ARG


def test_binding_shares_the_process_standard_library(ra):
    """The extension uses the process's libstdc++ (a copy of its own crashed when an
    error's numbers were printed on a machine with a GPU), and a wrong call says so."""
    import os
    import subprocess
    binding = ra._load_binding()
    path = os.path.join(os.path.dirname(ra.LIB_PATH), "_torch_binding.so")
    assert os.path.samefile(binding.__file__, path)
    needed = subprocess.run(["readelf", "-d", path], capture_output=True, text=True, check=True).stdout
    assert "libstdc++.so" in needed
    with pytest.raises(TypeError, match="10 arguments, got 1"):
        binding.qk_norm_rope(None)
    with pytest.raises(ValueError, match="q must be a tensor"):
        ra.qk_norm_rope(None)


def test_swc_cache8_refuses(ra):
    for args in ((0, 1, 64, 4, 2), (1, 0, 64, 4, 2), (1, 1, 96, 4, 2), (1, 1, 64, 0, 2), (1, 1, 64, 4, 0)):
        with pytest.raises(ValueError):
            ra.SwcCache8(*args)
