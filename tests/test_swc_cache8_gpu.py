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
