"""SwcCache8's own bookkeeping (CPU only: the calls under it are stand-ins)."""
import pytest
import torch


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import static_sparse_attention_b200 as ra
    return ra


class Calls:
    """Stand-ins of the extension's functions: the appends they saw, and an attention
    that refuses a scale or an lse as the library does, or fails to launch."""

    def __init__(self, W):
        self.appended, self.launch_fails, self.W = [], False, W

    def qk_norm_rope(self, q, *rest):
        return q, None

    def cache8_append(self, k, v, k8, v8, ks, vs, frame, *rest):
        self.appended.append(frame)
        return 0

    def _refusal(self, held, scale, lse):
        assert 1 <= held <= self.W
        if lse is not None and lse.dim() != 3:
            raise ValueError("lse must be a contiguous fp32 tensor [B, H, nq] on the inputs' device")
        return 1 if scale is not None and not scale > 0 else None

    def cache8_attention_prepare(self, q, k8, v8, ks, vs, held, counts, scale, out, lse, workspace, stream):
        r = self._refusal(held, scale, lse)
        return (q if out is None else out, workspace) if r is None else r

    def cache8_attention(self, q, k8, v8, ks, vs, held, counts, scale, out, lse, workspace, stream):
        r = 3 if self.launch_fails else self._refusal(held, scale, lse)
        return (q if out is None else out) if r is None else r


@pytest.fixture
def cache(ra, monkeypatch):
    monkeypatch.setattr(ra, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(ra, "_refuse_capture", lambda stream: None)
    c = object.__new__(ra.SwcCache8)
    c.B, c.H, c.d, c.s, c.W = 1, 2, 64, 4, 2
    c.k8 = c.v8 = torch.zeros(1, 2, 8, 64)
    c.k_scale = c.v_scale = torch.zeros(1, 2, 2, 1)
    c.frames_seen, c._streams = 0, {0}
    c.calls = Calls(c.W)
    monkeypatch.setattr(ra, "_binding", c.calls)
    return c


def test_a_refused_step_feeds_nothing(ra, cache):
    """A step whose attention is refused appends no frame; the same step again is that
    frame, in its slot and at its position."""
    x, w = torch.zeros(1, 4, 2, 64), torch.ones(64)
    for seen in range(4):
        for bad, error in ((dict(lse=torch.zeros(3)), ValueError), (dict(scale=0.0), ra.RaError),
                           (dict(scale=-1.0), ra.RaError)):
            with pytest.raises(error):
                cache.step(x, x, x, w, w, **bad)
            assert cache.info == dict(frames_seen=seen, frames_held=min(seen, 2))
        assert cache.calls.appended == list(range(seen))
        cache.step(x, x, x, w, w)
        assert cache.calls.appended == list(range(seen + 1))


def test_a_step_that_fails_to_launch_is_the_same_frame_again(ra, cache):
    x, w = torch.zeros(1, 4, 2, 64), torch.ones(64)
    cache.step(x, x, x, w, w)
    cache.calls.launch_fails = True
    with pytest.raises(ra.RaError):
        cache.step(x, x, x, w, w)
    assert cache.frames_seen == 1
    cache.calls.launch_fails = False
    cache.step(x, x, x, w, w)
    assert cache.frames_seen == 2 and cache.calls.appended == [0, 1, 1]
