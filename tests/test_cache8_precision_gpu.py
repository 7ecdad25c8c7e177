"""How precisely the attention over the 8-bit ring holds P: ra_set_pv_precision reaches
it, and the default holds P as hi + lo over fewer than 4096 keys (up to four queries
always), as the library's other attention does."""
import math

import pytest
import torch

from tests import _gpu, _heads

pytestmark = pytest.mark.gpu


@pytest.fixture
def policy():
    ra = _gpu.ra()
    yield lambda value: ra.check(ra.ra_set_pv_precision(value), "ra_set_pv_precision")
    ra.ra_set_pv_precision(ra.RA_PV_AUTO)


LIVE = 32  # keys of weight in each ring


def _cancelling(B, H, d, s, W, nq, seed):
    """A ring whose outputs are small differences of large terms: the keys of weight
    come in neighbouring pairs with nearly the same score and opposite values.  Every
    other key lies 200 or more (base e) below them: its weight is 2^-288, exactly 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nk = s * W
    k = torch.randn(B, H, nk, d, generator=g, device="cuda").to(torch.float8_e4m3fn)
    v = torch.randn(B, H, nk, d, generator=g, device="cuda").to(torch.float8_e4m3fn)
    kb, vb = k.view(torch.uint8), v.view(torch.uint8)
    pairs = min(LIVE, nk) // 2
    first = torch.linspace(0, nk // 2 - 1, pairs, device="cuda").round().long() * 2
    kb[..., 0] = 0xFE  # -448 in channel 0
    kb[:, :, first, 0] = 0
    kb[:, :, first, 1] = torch.randint(0x30, 0x3F, (B, H, pairs), generator=g, device="cuda", dtype=torch.uint8)
    kb[:, :, first + 1] = kb[:, :, first]
    kb[:, :, first + 1, 1] += 1  # the next code
    vb[:, :, first + 1] = vb[:, :, first] ^ 0x80
    blocks = -(-s // 64)
    ks, vs = (torch.exp2(torch.randint(-1, 2, (B, H, W, blocks), generator=g, device="cuda").float()) for _ in range(2))
    q = torch.randn(B, H, nq, d, generator=g, device="cuda").mul(0.5)
    q[..., 0] = 24.0
    return q.bfloat16(), (k, v, ks, vs), pairs * 2


def _worst(q, ring, s, W, live, held_as):
    """Largest error of O in units of its bound, P off by `held_as` of itself:
      x = scale q.k of a key of weight: d + 8 fp32 roundings, e_x <= (d + 8) U32 scale sum |q_i k_i|
          (channel 0 adds an exact 0), P off by 2 e_x and 2^-20 (exponential, rescales);
      the sums: hi and lo of `live` keys, each addition off by at most 2 U32 (the tensor core
          may cut off) of the sum of magnitudes, the other keys' terms exactly 0;
      O's own rounding, BF16 of it."""
    ra = _gpu.ra()
    B, H, nq, d = q.shape
    k8, v8, ks, vs = ring
    o = ra.cache8_attention(q, *ring, W)
    assert ra.device_status() == ra.RA_OK
    k = (k8.double() * _heads.per_token(ks.double(), s))
    v = (v8.double() * _heads.per_token(vs.double(), s))
    x = q.double() @ k.transpose(2, 3) / math.sqrt(d)
    p = torch.softmax(x, -1)
    alive = p > 1e-30
    assert int(alive.sum(-1).max()) <= live and float((x - x.amax(-1, keepdim=True))[~alive].max() if live < s * W
                                                       else -300) < -200
    e = (q[..., 1:].double().abs() @ k[..., 1:].abs().transpose(2, 3) / math.sqrt(d) * (d + 8) * _heads.U32)
    e = torch.where(alive, e, 0).amax(-1, keepdim=True)
    want, size = p @ v, p @ v.abs()
    bound = want.abs() * _heads.BF16 + size * (held_as + 2 * e + 2.0 ** -20 + 4 * live * _heads.U32) + 1e-30
    return ((o.double() - want).abs() / bound).max().item()


PAIR = _heads.BF16 ** 2  # hi is off by BF16 of P at most, lo by BF16 of that

#           B, H, d, s, W, nq
SHORT = [
    (2, 3, 64, 1, 2, 1),           # two keys
    (2, 3, 128, 64, 4, 1),
    (2, 3, 64, 50, 4, 3),
    (2, 3, 128, 50, 4, 4),
    (2, 3, 64, 64, 5, 8),
    (2, 3, 128, 64, 5, 16),
    (2, 3, 64, 50, 40, 2),         # ranges that are joined
    (2, 3, 128, 50, 40, 7),
    (2, 3, 64, 50, 40, 13),
    (40, 37, 64, 64, 4, 3),        # heads enough for several waves of blocks
    (40, 37, 128, 64, 4, 6),
    (40, 37, 64, 64, 4, 5),
    (4, 74, 64, 64, 4, 40),        # many queries, one tile a block
    (4, 74, 128, 50, 4, 100),
    (4, 74, 64, 64, 4, 200),       # and two
    (4, 74, 128, 50, 4, 256),
    (1, 2, 64, 50, 40, 70),        # joined
    (1, 2, 128, 64, 63, 300),
]


@pytest.mark.parametrize("case", SHORT, ids=lambda c: "x".join(map(str, c)))
def test_few_keys_hold_p_as_a_pair(case, policy):
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W, nq = case
    q, ring, live = _cancelling(*case, seed=sum(case))
    assert s * W < 4096
    for value in (ra.RA_PV_AUTO, ra.RA_PV_SPLIT):
        policy(value)
        worst = _worst(q, ring, s, W, live, PAIR)
        assert worst <= 1, f"policy {value}: off by {worst:.3g} of the bound"
    policy(ra.RA_PV_BF16)
    assert _worst(q, ring, s, W, live, _heads.BF16) <= 1
    if nq > 4 and live > 2:  # the case tells the two apart
        assert _worst(q, ring, s, W, live, PAIR) > 1


@pytest.mark.parametrize("case", [(2, 3, 128, 1, 5000, 1), (2, 3, 64, 50, 100, 4), (2, 3, 128, 50, 100, 8),
                                  (2, 3, 64, 50, 100, 16), (1, 2, 128, 64, 70, 33), (1, 2, 64, 100, 60, 280)],
                         ids=lambda c: "x".join(map(str, c)))
def test_many_keys_hold_p_as_asked(case, policy):
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W, nq = case
    q, ring, live = _cancelling(*case, seed=sum(case))
    assert s * W >= 4096
    policy(ra.RA_PV_SPLIT)
    worst = _worst(q, ring, s, W, live, PAIR)
    assert worst <= 1, f"off by {worst:.3g} of the bound"
    for value in (ra.RA_PV_AUTO, ra.RA_PV_BF16):
        policy(value)
        assert _worst(q, ring, s, W, live, PAIR if nq <= 4 else _heads.BF16) <= 1
