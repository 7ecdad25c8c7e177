"""Which packed gradients qk_norm_rope_bwd takes (CPU only: addresses are made up and
never dereferenced; a call that passes every check ends at the launch, for want of a
GPU, with another status than a refusal)."""
import ctypes
import itertools

import pytest
import torch

MB = 1 << 20


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import static_sparse_attention_b200 as ra
    return ra


def _taken(ra, B, n, d, dq, dk):
    """dq, dk: (offset in elements, strides, heads) in one buffer."""
    rows = [ra.ra_head_rows(x, n * h * d, h * d, d, h, 0, w) for x, w, (_, _, h) in
            ((100 * MB, 9 * MB, dq), (200 * MB, 9 * MB + 4096, dk))]
    grads = [ra.ra_head_grads(dy, 300 * MB + 2 * at, *strides, dw) for dy, dw, (at, strides, _) in
             ((400 * MB, 24 * MB, dq), (500 * MB, 25 * MB, dk))]
    need = ra.ra_qk_norm_rope_bwd_workspace_bytes(d)
    st = ra.ra_qk_norm_rope_bwd(ctypes.byref(rows[0]), ctypes.byref(rows[1]), ctypes.byref(grads[0]),
                                ctypes.byref(grads[1]), B, n, d, None, 0, 1e-6, 26 * MB, need, None)
    if st == ra.RA_ERR_INVALID_ARG:
        return False
    assert st == ra.RA_ERR_CUDA, (st, ra.ra_last_error())  # no device here
    return True


def _elements(B, n, d, at, strides, heads):
    """Every element's place, sorted."""
    out = [at + b * strides[0] + i * strides[1] + h * strides[2] + c
           for b in range(B) for i in range(n) for h in range(heads) for c in range(0, d, 8)]
    return out


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses must not reach a GPU")


@needs_no_gpu
@pytest.mark.parametrize("B,n,d,dq,dk", [
    # the next batch element's dq begins where this one's last dk ends
    (2, 2, 64, (0, (192, 128, 64), 1), (64, (192, 128, 64), 1)),
    # dk of a token's second head is dq of the next token's
    (1, 2, 64, (0, (768, 192, 128), 2), (64, (768, 192, 128), 2)),
    # the same rows of a head-major buffer, one token on
    (1, 3, 64, (0, (1024, 64, 512), 2), (64, (1024, 64, 512), 2)),
    # the slots of a token, and batch elements that begin inside the last token's
    (2, 3, 64, (0, (704, 256, 64), 1), (192, (704, 256, 64), 1)),
])
def test_packed_gradients_that_overlap_are_refused(ra, B, n, d, dq, dk):
    shared = set(_elements(B, n, d, *dq)) & set(_elements(B, n, d, *dk))
    assert shared, "the case is one of overlap"
    assert not _taken(ra, B, n, d, dq, dk)
    assert b"alias" in ra.ra_last_error()
    assert not _taken(ra, B, n, d, dk, dq)


@needs_no_gpu
@pytest.mark.parametrize("B,n,d,dq,dk", [
    (2, 5, 64, (0, (5 * 448, 448, 64), 3), (192, (5 * 448, 448, 64), 2)),         # [B, n, 3 + 2 + 2, d]
    (2, 5, 128, (0, (5 * 1152, 1152, 384), 3), (128, (5 * 1152, 1152, 384), 3)),  # [B, n, H, 3, d]
    (2, 5, 64, (0, (6 * 320, 64, 320), 3), (960, (6 * 320, 64, 320), 3)),         # [B, 2 H, n, d]
    (2, 1, 64, (0, (384, 64, 64), 3), (192, (384, 64, 64), 3)),                   # one token
    (1, 2, 64, (64, (0, 128, 64), 1), (0, (0, 128, 64), 1)),                      # dk first
])
def test_packed_gradients_of_their_own_are_taken(ra, B, n, d, dq, dk):
    assert not set(_elements(B, n, d, *dq)) & set(_elements(B, n, d, *dk))
    assert _taken(ra, B, n, d, dq, dk)


@needs_no_gpu
def test_no_overlap_is_taken(ra):
    """Over all small strides: what is taken shares no element (the converse need not
    hold: a layout that is no packing is refused)."""
    B, n, d, H, taken = 2, 2, 64, 2, 0
    steps = (64, 128, 192, 256, 384, 512, 768)
    for strides in itertools.product(steps, repeat=3):
        for at in (64, 128, 256, 384):
            dq, dk = (0, strides, H), (at, strides, H)
            if _taken(ra, B, n, d, dq, dk):
                taken += 1
                parts = _elements(B, n, d, *dq) + _elements(B, n, d, *dk)
                assert len(set(parts)) == len(parts), (strides, at)
    assert taken > 20
