"""Every kernel of the attention over the 8-bit ring, each named and asked for: which one
a call runs depends on its sizes (a few queries, or many over few keys and heads, take
the kernel of few queries), so each case here checks that it reaches the one it means."""
import ctypes
import math

import pytest
import torch

from tests import _gpu, _heads
from tests.test_cache8_gpu import _check, _reference, _ring, _values

pytestmark = pytest.mark.gpu

ROWS, ROWS_AHEAD, ONE_TILE, TWO_TILES = range(4)


def _plan(B, H, d, nq, s, W, held):
    ra = _gpu.ra()
    kernel, ranges = ctypes.c_int(-1), ctypes.c_int(-1)
    ra.check(ra.ra_cache8_attention_plan(B, H, d, nq, s, W, held, ctypes.byref(kernel), ctypes.byref(ranges)), "plan")
    return kernel.value, ranges.value


#         kernel, B, H, nq, held (of 64-token frames), joined
SIZES = [
    (ROWS, 30, 37, 1, 9, False),
    (ROWS, 30, 37, 6, 9, False),
    (ROWS_AHEAD, 2, 3, 2, 8, False),
    (ROWS_AHEAD, 2, 3, 16, 40, True),
    (ONE_TILE, 4, 38, 100, 9, False),
    (ONE_TILE, 2, 3, 40, 30, True),
    (TWO_TILES, 4, 74, 256, 9, False),
    (TWO_TILES, 2, 20, 200, 60, True),
]


def _size(size, d):
    kernel, B, H, nq, held, joined = size
    got = _plan(B, H, d, nq, 64, held + 1, held)
    assert got[0] == kernel and (got[1] > 1) == joined, got
    return B, H, nq, held, held + 1


sizes = pytest.mark.parametrize("size", SIZES, ids=lambda x: f"kernel{x[0]}-{x[3]}{'-joined' if x[5] else ''}")
channels = pytest.mark.parametrize("d", [64, 128])


@channels
@sizes
def test_counts(size, d):
    """Batch elements of unequal lengths: none, one, at the ends of groups, steps and ranges."""
    _gpu.need_gpu()
    B, H, nq, held, W = _size(size, d)
    n = held * 64
    counts = [0, 1, 15, 17, 63, 64, 65, n // 2, n - 1, n, n + 5, -1]
    counts = (counts[::-1] + counts * 2)[:B] if B > 2 else [n - 1, 65]
    ring, guards = _ring(B, H, d, 64, W, seed=B + nq)
    q = torch.randn(B, H, nq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    if B * H * nq * n * d > 2e9:  # the reference is on the CPU: a few heads of it
        _check_heads(q, ring, held, counts, (0, H // 2, H - 1))
    else:
        _check(q, ring, 64, held, (counts + [n] * B)[:B], what=str(size))
    _gpu.check_canaries(*guards, what="the ring is only read")


def _check_heads(q, ring, held, counts, heads, scale=None):
    ra = _gpu.ra()
    B, H, nq, d = q.shape
    n = held * 64
    counts = (counts + [n] * B)[:B]
    lse = torch.full((B, H, nq), 7.0, device="cuda")
    o = ra.cache8_attention(q, *ring, held, key_counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), lse=lse,
                            scale=scale)
    assert ra.device_status() == ra.RA_OK
    assert not bool(torch.isnan(o).any()) and not bool(torch.isnan(lse).any())
    real = [min(max(c, 0), n) for c in counts]
    for h in heads:
        at = slice(h, h + 1)
        k8, v8, ks, vs = (t[:, at] for t in ring)
        want, want_lse, ob, lb = _reference(q[:, at], k8, v8, ks, vs, 64, real, scale or 1 / math.sqrt(d))
        off = ((o[:, at].double().cpu() - want).abs() / ob).max()
        assert off <= 1, f"head {h}: o off by {off:.3g} of the bound"
        got = lse[:, at].double().cpu()
        empty = torch.isinf(want_lse)
        assert torch.equal(got[empty], want_lse[empty])
        off = ((got - want_lse).abs() / lb)[~empty].max()
        assert off <= 1, f"head {h}: lse off by {off:.3g} of the bound"


@channels
@sizes
def test_no_frames(size, d):
    _gpu.need_gpu()
    ra = _gpu.ra()
    kernel, B, H, nq, held, joined = size
    if kernel != ROWS_AHEAD:
        B, H = max(B, 4), max(H, 74)
    assert _plan(B, H, d, nq, 64, 2, 0) == (kernel, 1)
    ring, _ = _ring(B, H, d, 64, 2)
    lse = torch.zeros(B, H, nq, device="cuda")
    o = ra.cache8_attention(torch.randn(B, H, nq, d, device="cuda").bfloat16(), *ring, 0, lse=lse)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


CODES = [c for c in range(256) if c & 127 != 127]


@sizes
@pytest.mark.parametrize("exponent", [-110, -9, 0, 7, 8, 60, 110])
def test_every_code_of_v_at_every_scale(size, exponent):
    """One key of weight (the count is 1): the output is its value, code * scale, exactly.
    The other frames' scales are small, so that scales of one and of two factors meet in
    a step."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    d = 128
    B, H, nq, held, W = _size(size, d)
    k8 = torch.zeros(B, H, W * 64, d, dtype=torch.uint8, device="cuda")
    v8 = torch.full_like(k8, 0x7E)
    codes = torch.tensor(CODES, dtype=torch.uint8, device="cuda")
    v8[:, 0::2, 0], v8[:, 1::2, 0] = codes[:128], codes[126:]
    ks, vs = (torch.ones(B, H, W, 1, device="cuda") for _ in range(2))
    vs.mul_(2.0 ** -20)
    vs[:, :, 0] = 2.0 ** exponent
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
    o = ra.cache8_attention(q, k8.view(torch.float8_e4m3fn), v8.view(torch.float8_e4m3fn), ks, vs, held, key_counts=ones)
    for head, part in ((0, codes[:128]), (1, codes[126:])):
        want = (part.view(torch.float8_e4m3fn).double() * 2.0 ** exponent).to(torch.bfloat16)
        assert torch.equal(o[:, head::2], want.expand(B, len(range(head, H, 2)), nq, d))


@sizes
@pytest.mark.parametrize("exponent", [-110, -9, 0, 7, 8])
def test_every_code_of_k_at_every_scale(size, exponent):
    """The lse of a single key is its score: one code against a one-hot query."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    d = 128
    B, H, nq, held, W = _size(size, d)
    k8 = torch.zeros(B, H, W * 64, d, dtype=torch.uint8, device="cuda")
    codes = torch.tensor(CODES, dtype=torch.uint8, device="cuda")
    k8[:, 0::2, 0], k8[:, 1::2, 0] = codes[:128], codes[126:]
    ks, vs = (torch.ones(B, H, W, 1, device="cuda") for _ in range(2))
    ks[:, :, 0] = 2.0 ** exponent
    counts = torch.ones(B, dtype=torch.int32, device="cuda")
    for shift in range(0, 128, 43 if nq > 4 else 1):
        at = (torch.arange(nq, device="cuda") * 3 + shift) % d  # query i asks for channel at[i]
        q = torch.zeros(B, H, nq, d, device="cuda", dtype=torch.bfloat16)
        q[:, :, torch.arange(nq), at] = 1
        lse = torch.empty(B, H, nq, device="cuda")
        ra.cache8_attention(q, k8.view(torch.float8_e4m3fn), k8.view(torch.float8_e4m3fn), ks, vs, held,
                            key_counts=counts, scale=1.0, lse=lse)
        for head, part in ((0, codes[:128]), (1, codes[126:])):
            want = (part.view(torch.float8_e4m3fn).double() * 2.0 ** exponent)[at].expand(B, len(range(head, H, 2)), nq)
            # base 2 and back: two fp32 roundings and the constants' own
            assert torch.allclose(lse[:, head::2].double(), want, rtol=4 * _heads.U32, atol=1e-37)


@channels
@sizes
def test_large_scales(size, d):
    """Scales above 2^7 (two factors) and below in one step, in K and in V: block b of K has
    2^(b mod 3 * 4), its codes small in proportion; V's 2^(8 b mod 24)."""
    _gpu.need_gpu()
    B, H, nq, held, W = _size(size, d)
    (k8, v8, ks, vs), _ = _ring(B, H, d, 64, W, seed=7)
    b = torch.arange(W, device="cuda")
    ks.copy_(torch.exp2(-9.0 + 0 * b)[None, None, :, None].expand_as(ks))
    ks[:, :, 1::3] = 2.0 ** 8
    kb = k8.view(torch.uint8).view(B, H, W, 64, d)
    kb[:, :, 1::3] = (kb[:, :, 1::3] & 0x80) | (kb[:, :, 1::3] & 7)  # subnormal codes, up to 7 * 2^-9
    vs.copy_(torch.exp2((8 * b % 24).float())[None, None, :, None].expand_as(vs))
    q = (torch.randn(B, H, nq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) / 8).bfloat16()
    _check_heads(q, (k8, v8, ks, vs), held, [], (0, H - 1))


@channels
@sizes
def test_scales_that_are_no_powers_of_two(size, d):
    """Another quantiser's scales: code * scale is rounded to bf16 at most three times."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, nq, held, W = _size(size, d)
    (k8, v8, ks, vs), _ = _ring(B, H, d, 64, W, seed=8)
    ks.mul_(1.3)
    vs.mul_(0.7)
    q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
    o = ra.cache8_attention(q, k8, v8, ks, vs, held)
    for h in (0, H - 1):
        at, n = slice(h, h + 1), held * 64
        k, v = _values(k8[:, at], ks[:, at], 64)[:, :, :n], _values(v8[:, at], vs[:, at], 64)[:, :, :n]
        qh = q[:, at].double().cpu()
        x = qh @ k.transpose(2, 3) / math.sqrt(d)
        p = torch.softmax(x, -1)
        off = 3 * _heads.BF16
        e = (qh.abs() @ k.abs().transpose(2, 3) / math.sqrt(d)).amax(-1, keepdim=True) * off
        bound = (p @ v).abs() * _heads.BF16 + (p @ v.abs()) * (off + _heads.BF16 + torch.expm1(2 * e))
        assert bool(((o[:, at].double().cpu() - p @ v).abs() <= bound).all())


@channels
@sizes
def test_what_is_not_finite_stays_where_it_is_read(size, d):
    """A NaN scale poisons the heads that attend to its block, not one whose count ends
    before it nor one where it lies behind the frames held; a NaN query poisons its row."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, nq, held, W = _size(size, d)
    (k8, v8, ks, vs), _ = _ring(B, H, d, 64, W, seed=9)
    ks[0, 1, 2] = math.nan
    vs[0, 2, 5] = math.nan
    vs[1, 0, held] = math.nan       # not held
    ks[1, 1, held - 1] = math.nan   # behind the count
    vs[1, 2, held - 1] = math.nan
    q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
    row = nq // 2
    q[1, 1, row, 3] = math.nan
    counts = torch.full((B,), held * 64, dtype=torch.int32, device="cuda")
    counts[1] = (held - 1) * 64
    lse = torch.empty(B, H, nq, device="cuda")
    o = ra.cache8_attention(q, k8, v8, ks, vs, held, key_counts=counts, lse=lse)
    assert ra.device_status() == ra.RA_OK
    bad, scores = torch.zeros(B, H, nq, dtype=torch.bool, device="cuda"), torch.zeros(B, H, nq, dtype=torch.bool, device="cuda")
    bad[0, 1], bad[0, 2], bad[1, 1, row] = True, True, True
    scores[0, 1], scores[1, 1, row] = True, True
    assert torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), scores)
    counts[0] = 2 * 64  # up to the first, not into it
    q[1, 1, row, 3] = 0
    assert not bool(torch.isnan(ra.cache8_attention(q, k8, v8, ks, vs, held, key_counts=counts)).any())


@pytest.mark.parametrize("B,H,d,grid,W,f", [(1, 6, 128, (13, 20), 4, 7), (2, 40, 64, (8, 9), 3, 5)], ids=lambda x: str(x))
def test_stream(B, H, d, grid, W, f):
    """Frames through SwcCache8 as a model feeds them, sizes at which the tensor-memory
    kernel attends."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    s = grid[0] * grid[1]
    g = torch.Generator(device="cuda").manual_seed(s)
    q, k, v = torch.randn(B, f * s, 3 * H, d, generator=g, device="cuda").bfloat16().split(H, dim=2)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = ra.rope3d(f, *grid, d)
    cache = ra.SwcCache8(B, H, d, s, W)
    for i in range(f):
        at, held = slice(i * s, (i + 1) * s), min(i + 1, W)
        assert i < 1 or _plan(B, H, d, s, s, W, held)[0] >= ONE_TILE
        lse = torch.empty(B, H, s, device="cuda")
        o = cache.step(q[:, at], k[:, at], v[:, at], wq, wk, rope, 1e-6, lse=lse)
        yq, _ = ra.qk_norm_rope(q[:, at], None, wq, rope=rope, frame0=i, eps=1e-6)
        for h in (0, H - 1):
            one = slice(h, h + 1)
            want, want_lse, ob, lb = _reference(yq[:, one], *(t[:, one, :held * s] for t in (cache.k8, cache.v8)),
                                                *(t[:, one, :held] for t in (cache.k_scale, cache.v_scale)), s,
                                                [held * s] * B, 1 / math.sqrt(d))
            assert bool(((o[:, one].double().cpu() - want).abs() <= ob).all())
            assert bool(((lse[:, one].double().cpu() - want_lse).abs() <= lb).all())
    assert ra.device_status() == ra.RA_OK
