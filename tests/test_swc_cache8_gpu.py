"""SwcCache8 as an object: the streams it is used on, and calls that it refuses."""
import pytest
import torch

from tests import _gpu

pytestmark = pytest.mark.gpu

SLEEP = 40_000_000  # clocks: 20 ms or more


def _frames(B, H, d, s, n, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [tuple(torch.randn(B, s, H, d, generator=g, device="cuda").bfloat16() for _ in range(3)) for _ in range(n)]


def _bits(cache):
    return [t.view(torch.uint8).clone() for t in cache._ring]


@pytest.mark.parametrize("context", [False, True], ids=["argument", "current"])
def test_steps_on_another_stream_than_the_creating_one(context):
    """The ring's first fills are on the creating stream, which may be far behind: a
    step on another stream must come after them."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 2, 64, 70, 3
    frames = _frames(B, H, d, s, 4)
    plain = ra.SwcCache8(B, H, d, s, W)
    want = [plain.step(*f) for f in frames]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SLEEP)
    cache = ra.SwcCache8(B, H, d, s, W)
    if context:
        with torch.cuda.stream(side):
            got = [cache.step(*f) for f in frames]
    else:
        got = [cache.step(*f, stream=side) for f in frames]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(_bits(cache), _bits(plain)):
        assert torch.equal(a, b)


def test_the_ring_outlives_its_object_until_the_stream_is_done():
    """Memory of a ring dropped while another stream still works on it is not handed
    out before that work is done."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 2, 64, 256, 8
    frames = _frames(B, H, d, s, 2)
    plain = ra.SwcCache8(B, H, d, s, W)
    want = [plain.step(*f) for f in frames]
    side = torch.cuda.Stream()
    cache = ra.SwcCache8(B, H, d, s, W)
    torch.cuda.synchronize()
    places = {t.data_ptr() for t in cache._ring}
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = [cache.step(*f, stream=side) for f in frames]
    del cache
    taken = [torch.full((B, H, W * s, d), 0x7E, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not places & {t.data_ptr() for t in taken}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_refused_step_leaves_the_ring_as_it_was():
    """Whatever a step refuses, the ring keeps every bit and the frame's number; the
    stream goes on as if the refused step had not been."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 2, 64, 70, 3
    frames = _frames(B, H, d, s, 5)
    w = torch.ones(d, device="cuda")
    rope = ra.rope3d(5, 7, 10, d)
    plain, cache = ra.SwcCache8(B, H, d, s, W), ra.SwcCache8(B, H, d, s, W)
    inside = cache.k8.view(torch.uint8).view(-1)[:2 * B * H * s * d].view(torch.bfloat16).view(B, H, s, d)
    for i, (q, k, v) in enumerate(frames):
        before = _bits(cache)
        for bad, error in ((dict(lse=torch.empty(B, H, s + 1, device="cuda")), ValueError),
                           (dict(out=torch.empty(B, H, s, d, device="cuda")), ValueError),
                           (dict(out=inside), ra.RaError),
                           (dict(scale=0.0), ra.RaError), (dict(scale=float("inf")), ra.RaError),
                           (dict(eps=0.0), ra.RaError), (dict(k_weight=w[:8]), ValueError)):
            with pytest.raises(error):
                cache.step(q, k, v, **{**dict(q_weight=w, k_weight=w, rope=rope), **bad})
        with pytest.raises(ValueError):
            cache.step(q, k, v.float(), w, w, rope)
        assert cache.info == dict(frames_seen=i, frames_held=min(i, W))
        assert all(torch.equal(a, b) for a, b in zip(before, _bits(cache)))
        assert torch.equal(cache.step(q, k, v, w, w, rope), plain.step(q, k, v, w, w, rope))
    with pytest.raises(ra.RaError):  # frame 5 of a table of 5
        cache.step(q, k, v, w, w, rope)
    assert cache.frames_seen == 5
