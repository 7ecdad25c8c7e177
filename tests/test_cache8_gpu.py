"""The 8-bit key/value ring against 64-bit forms (tests/_heads.py): what an append
writes (codes, scales, the slots of other frames) and attention over it."""
import math

import pytest
import torch

from tests import _gpu, _heads

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _ring(B, H, d, s, W, seed=0):
    """Random codes (none of NaN) and power-of-two scales in canary bands: (k8, v8, k_scale, v_scale), guards"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = -(-s // 64)
    guards, out = [], []
    for _ in range(2):
        band = _gpu.Guarded((B * H * W * s * d // 2,), torch.bfloat16)  # two codes an element
        code = band.t.view(torch.uint8).view(B, H, W * s, d)
        code.copy_(torch.randint(0, 127, code.shape, generator=g, device="cuda", dtype=torch.uint8)
                   + 128 * torch.randint(0, 2, code.shape, generator=g, device="cuda", dtype=torch.uint8))
        guards.append(band)
        out.append(code.view(torch.float8_e4m3fn))
    for _ in range(2):
        band = _gpu.Guarded((B, H, W, blocks), torch.float32)
        band.t.copy_(torch.exp2(torch.randint(-12, -6, band.t.shape, generator=g, device="cuda").float()))
        guards.append(band)
        out.append(band.t)
    return out, guards


def _values(code, scale, s):
    """fp64 values [B, H, W * s, d] on the CPU"""
    return code.float().double().cpu() * _heads.per_token(scale.double().cpu(), s)


# ------------------------------------------------------------------------ append
#        B, H, d, grid, W, frames, frame
APPENDS = [
    (1, 1, 64, (1, 1), 1, 1, 0),
    (2, 3, 128, (1, 1), 7, 1, 40),       # single tokens: a scale each
    (2, 3, 64, (1, 1), 5, 5, 3),         # wraps around the ring's end
    (1, 2, 128, (3, 5), 4, 2, 7),        # fewer rows than a pass
    (1, 2, 64, (4, 16), 3, 1, 2),        # exactly one block
    (1, 3, 128, (5, 13), 3, 3, 1),       # one row over a block
    (2, 2, 64, (11, 17), 2, 1, 9),
    (1, 2, 128, (16, 24), 4, 3, 5),
]


@pytest.mark.parametrize("norm,rotated,packed", [(True, True, True), (False, False, False), (True, False, True),
                                                 (False, True, False)], ids=["norm+rope", "plain", "norm", "rope"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "x".join(str(x) for x in c))
def test_append(case, norm, rotated, packed):
    """V's codes and scales are exact (a bf16 value needs no arithmetic before the
    rounding); K's scale may only differ where fp32 puts the block's largest value
    across the border, and its values by one code step where it puts a value across
    a rounding border; slots of other frames keep every bit."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, (gh, gw), W, frames, frame = case
    s = gh * gw
    n = frames * s
    g = torch.Generator(device="cuda").manual_seed(n + H)
    if packed:
        _, k, v = torch.randn(B, n, 3 * H, d, generator=g, device="cuda").bfloat16().split(H, dim=2)
    else:
        k, v = (torch.randn(B, H, n, d, generator=g, device="cuda").mul(m).bfloat16().transpose(1, 2)
                for m in (1e-3, 300.0))
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16() if norm else None
    rope = ra.rope3d(frame + frames, gh, gw, d) if rotated else None
    (k8, v8, ks, vs), guards = _ring(B, H, d, s, W, seed=5)
    before = [t.clone() for t in (k8.view(torch.uint8), v8.view(torch.uint8), ks, vs)]
    ra.cache8_append(k, v, k8, v8, ks, vs, frame, w, rope=rope, eps=EPS)
    _gpu.check_canaries(*guards, what="append")
    slots = [(frame + j) % W for j in range(frames)]
    rows = torch.cat([torch.arange(x * s, (x + 1) * s) for x in slots])
    k64, bound = _heads.norm_rope(k, w, rope, frame, EPS)
    bound = bound - k64.abs() * _heads.BF16  # not rounded to bf16 on the way
    if not norm and not rotated:
        bound = torch.zeros_like(bound)
    for name, x, err, code, scale in (("k", k64, bound, k8, ks), ("v", v.double().cpu().transpose(1, 2), None, v8, vs)):
        want = _heads.block_scales(x, s)
        got = scale[:, :, slots].double().cpu()
        unit = _heads.per_token(got, s)
        values = code.float().double().cpu()[:, :, rows]
        if err is None or not bool(err.any()):
            assert torch.equal(got, want), f"{name} scales"
            assert torch.equal(values, _heads.e4m3(x / unit)), f"{name} codes"
            continue
        low, high = _heads.block_scales(x.abs() - err, s), _heads.block_scales(x.abs() + err, s)
        assert bool(((got >= torch.minimum(low, want)) & (got <= torch.maximum(high, want))).all()), f"{name} scales"
        low, high = _heads.e4m3((x - err) / unit), _heads.e4m3((x + err) / unit)
        assert bool(((values >= low) & (values <= high)).all()), f"{name} codes"
        # the bounds leave one code to nearly every value: one in 16 bf16 values, which an unturned channel still is
        # (position 0), lies on a tie of e4m3, whose 4 significant bits drop 4 of its 8
        assert float((low != high).double().mean()) < 2 / 16, "the bounds say something"
    others = [x for x in range(W) if x not in slots]
    rest = torch.cat([torch.arange(x * s, (x + 1) * s) for x in others]).cuda() if others else None
    if others:
        for t, b in zip((k8.view(torch.uint8), v8.view(torch.uint8)), before):
            assert torch.equal(t[:, :, rest], b[:, :, rest])
        for t, b in zip((ks, vs), before[2:]):
            assert torch.equal(t[:, :, others], b[:, :, others])


def test_append_at_the_borders():
    """Magnitudes on both sides of 448 * 2^k, subnormal codes, ties, zeros, the
    smallest and largest bf16 numbers, infinities and NaN."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 1, 64, 1, 16
    x = torch.zeros(B, W, H, d)
    x[0, 0, 0, 0] = 448.0                     # scale 1, the top code
    x[0, 1, 0, 0] = 450.0                     # bf16 above it: scale 2
    x[0, 2, 0, :4] = torch.tensor([256.0, 17.0, 19.0, -21.0])  # ties between codes of scale 1
    x[0, 3, 0, :3] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10])  # half a subnormal step: a tie to 0, one to 2
    x[0, 4, 0, 0] = 2.0 ** -130               # far below: scale 2^-126
    x[0, 5, 0, :2] = torch.tensor([3.3e38, -1.0])
    x[0, 6, 0, 0] = 2.0 ** -126
    x[0, 8, 0, 3] = float("inf")
    x[0, 9, 0, 3] = float("nan")
    x[0, 10, 0, :2] = torch.tensor([-448.0 * 2 ** 30, 2.0 ** 20])
    x = x.bfloat16().cuda()
    (k8, v8, ks, vs), _ = _ring(B, H, d, s, W)
    ra.cache8_append(x, x, k8, v8, ks, vs, 0)
    want = x.double().cpu().transpose(1, 2)
    fine = torch.isfinite(want).all(-1)[0, 0]
    scale = _heads.block_scales(torch.nan_to_num(want, 0, 0, 0), s)[..., 0]
    assert torch.equal(k8.view(torch.uint8), v8.view(torch.uint8)) and torch.equal(ks[0, 0, fine.cuda()], vs[0, 0, fine.cuda()])
    assert torch.equal(ks[0, 0, :, 0].double().cpu()[fine], scale[0, 0][fine])
    assert bool(torch.isnan(ks[0, 0, :, 0].cpu()[~fine]).all()) and int((~fine).sum()) == 2
    got = k8.float().double().cpu()
    assert torch.equal(got[0, 0][fine], _heads.e4m3(want / scale[..., None])[0, 0][fine])
    assert bool((got[0, 0][~fine] == 0).all())


# --------------------------------------------------------------------- attention
def _reference(q, k8, v8, ks, vs, s, counts, scale):
    """o, lse and the bounds of a kernel that multiplies exact bf16 operands into fp32
    sums and rounds P (and O at the end) to bf16:
      x = scale q.k: the products are exact, d + 8 fp32 roundings of partial sums give
          |dx| <= (d + 8) U32 * scale * sum |q_i k_i| = e_x, so P is off by a factor of e^(2 e_x)
          and 2^-20 more (the exponential's 2 units, the running sums' rescales);
      o: P's own rounding BF16 and the fp32 sums over the keys (n U32 of the sum of
          magnitudes), then the rounding of o: BF16 |o|."""
    B, H, nq, d = q.shape
    k, v = _values(k8, ks, s), _values(v8, vs, s)
    o, lse, ob, lb = [], [], [], []
    for b in range(B):
        n = counts[b]
        x = q[b].double().cpu() @ k[b, :, :n].transpose(1, 2) * scale
        e = q[b].double().cpu().abs() @ k[b, :, :n].abs().transpose(1, 2) * scale * (d + 8) * _heads.U32
        e = e.amax(-1, keepdim=True) if n else torch.zeros(H, nq, 1, dtype=torch.float64)
        z = torch.logsumexp(x, -1, keepdim=True) if n else torch.full((H, nq, 1), -math.inf, dtype=torch.float64)
        p = torch.exp(x - z) if n else x
        out = p @ v[b, :, :n]
        size = p @ v[b, :, :n].abs()
        o.append(out)
        lse.append(z[..., 0])
        ob.append(out.abs() * _heads.BF16 + size * (_heads.BF16 + 2 * e + 2.0 ** -20 + 2 * n * _heads.U32) + 1e-30)
        lb.append((e + 2.0 ** -20 + n * _heads.U32)[..., 0] + z.abs().nan_to_num(0, 0, 0)[..., 0] * 4 * _heads.U32)
    return (torch.stack(t) for t in (o, lse, ob, lb))


def _check(q, ring, s, held, counts=None, scale=None, what=""):
    ra = _gpu.ra()
    B, H, nq, d = q.shape
    k8, v8, ks, vs = ring
    go, gl = _gpu.Guarded((B, H, nq, d), torch.bfloat16), _gpu.Guarded((B, H, nq), torch.float32)
    dev = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    ra.cache8_attention(q, k8, v8, ks, vs, held, key_counts=dev, scale=scale, out=go.t, lse=gl.t)
    assert ra.device_status() == ra.RA_OK
    _gpu.check_canaries(go, gl, what=what)
    n = held * s
    real = [n] * B if counts is None else [min(max(c, 0), n) for c in counts]
    o, lse, ob, lb = _reference(q, k8, v8, ks, vs, s, real, 1 / math.sqrt(d) if scale is None else scale)
    got, got_lse = go.t.double().cpu(), gl.t.double().cpu()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    off = ((got - o).abs() / ob).max().item()
    assert off <= 1, f"{what}: o off by {off:.3g} of the bound"
    empty = torch.isinf(lse)
    assert torch.equal(got_lse[empty], lse[empty]), what
    off = ((got_lse - lse).abs() / lb)[~empty]
    assert off.numel() == 0 or off.max() <= 1, f"{what}: lse off by {off.max().item():.3g} of the bound"
    assert bool((got[empty] == 0).all())


#           B, H, d, s, W, held, nq
ATTENDS = [
    (1, 1, 64, 1, 1, 1, 1),          # one key
    (2, 3, 128, 1, 5, 5, 1),         # fewer keys than a group
    (1, 2, 64, 1, 300, 300, 1),      # single tokens, a scale each
    (2, 2, 128, 1, 4099, 4099, 1),   # the range splits, and ends inside a group
    (1, 3, 64, 7, 60, 41, 2),
    (1, 2, 128, 65, 9, 7, 16),       # blocks of 64 and of 1 alternate
    (1, 2, 64, 100, 12, 12, 17),     # one query over a tile of 16
    (2, 1, 128, 37, 30, 30, 40),
    (1, 2, 128, 64, 40, 33, 127),
    (1, 2, 64, 130, 6, 5, 128),
    (2, 2, 128, 130, 6, 5, 129),
    (1, 1, 128, 256, 9, 8, 256),
    (1, 2, 64, 200, 16, 16, 333),
    (1, 1, 64, 1560, 3, 2, 700),
    (1, 1, 128, 1, 20011, 20011, 3),
]


@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "x".join(str(x) for x in c))
def test_attention(case):
    _gpu.need_gpu()
    B, H, d, s, W, held, nq = case
    ring, guards = _ring(B, H, d, s, W, seed=sum(case))
    q = torch.randn(B, H, nq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    _check(q, ring, s, held, what=str(case))
    _check(q * 8, ring, s, held, scale=0.5, what=f"{case}, peaked")
    _gpu.check_canaries(*guards, what="the ring is only read")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 5, 16, 40, 130, 300])
def test_attention_of_a_ragged_batch(nq, d):
    """Counts of zero, one, inside and at the ends of blocks, tiles and splits, below
    zero and beyond the rows held (both clamped)."""
    _gpu.need_gpu()
    s, W, held = 77, 30, 27
    counts = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 1000, held * s - 1, held * s, 10 ** 9, -3]
    ring, _ = _ring(len(counts), 2, d, s, W, seed=nq)
    q = torch.randn(len(counts), 2, nq, d, device="cuda").bfloat16()
    _check(q, ring, s, held, counts, what=f"ragged, nq={nq}")


def test_attention_of_whole_frames():
    """Frames of 1560 tokens, 40 heads: every block walks all 98 steps of keys (its
    rings turn over many times) and a tile of 24 queries is left; two heads checked."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 40, 128, 1560, 5
    (k8, v8, ks, vs), _ = _ring(B, H, d, s, W, seed=4)
    q = torch.randn(B, H, s, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16()
    lse = torch.empty(B, H, s, device="cuda")
    o = ra.cache8_attention(q, k8, v8, ks, vs, 4, lse=lse)
    assert ra.device_status() == ra.RA_OK
    for h in (0, 39):
        at = slice(h, h + 1)
        want, want_lse, ob, lb = _reference(q[:, at], k8[:, at, :4 * s], v8[:, at, :4 * s], ks[:, at, :4], vs[:, at, :4], s,
                                            [4 * s], 1 / math.sqrt(d))
        assert bool(((o[:, at].double().cpu() - want).abs() <= ob).all())
        assert bool(((lse[:, at].double().cpu() - want_lse).abs() <= lb).all())


def test_scales_that_are_no_powers_of_two():
    """Another quantiser's scales: code * scale rounded to bf16 (of K in the product's
    order), so a value is off by at most three bf16 roundings."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 2, 64, 70, 4
    (k8, v8, ks, vs), _ = _ring(B, H, d, s, W, seed=8)
    ks.mul_(1.3)
    vs.mul_(0.7)
    for nq in (3, 200):
        q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
        o = ra.cache8_attention(q, k8, v8, ks, vs, W)
        k, v = _values(k8, ks, s), _values(v8, vs, s)
        x = q.double().cpu() @ k.transpose(2, 3) / math.sqrt(d)
        p = torch.softmax(x, -1)
        off = 3 * _heads.BF16
        e = (q.double().cpu().abs() @ k.abs().transpose(2, 3) / math.sqrt(d)).amax(-1, keepdim=True) * off
        bound = (p @ v).abs() * _heads.BF16 + (p @ v.abs()) * (off + _heads.BF16 + torch.expm1(2 * e))
        assert bool(((o.double().cpu() - p @ v).abs() <= bound).all())


def test_python_refusals():
    """Tensors of the wrong type, shape, layout or device are refused before any launch."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 2, 2, 64, 10, 3
    ring, _ = _ring(B, H, d, s, W)
    k8, v8, ks, vs = ring
    q = torch.randn(B, H, 4, d, device="cuda").bfloat16()
    x = torch.randn(B, s, H, d, device="cuda").bfloat16()
    counts = torch.zeros(B, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(q=q.transpose(1, 2)), dict(q=q[..., :32]),
                dict(k8=k8.view(torch.uint8)), dict(v8=v8[:, :, :-1]), dict(ks=ks.double()), dict(vs=vs[:, :, :2]),
                dict(ks=ks[:, :, :2]), dict(counts=counts.long()), dict(counts=counts[:1]), dict(counts=counts.cpu()),
                dict(out=torch.empty(B, H, 4, d, device="cuda")), dict(lse=torch.empty(B, H, 5, device="cuda")),
                dict(lse=torch.empty(B, H, 4, device="cuda", dtype=torch.bfloat16))):
        a = dict(q=q, k8=k8, v8=v8, ks=ks, vs=vs, counts=counts, out=None, lse=None)
        a.update(bad)
        with pytest.raises(ValueError):
            ra.cache8_attention(a["q"], a["k8"], a["v8"], a["ks"], a["vs"], W, key_counts=a["counts"], out=a["out"],
                                lse=a["lse"])
    for held in (-1, W + 1):
        with pytest.raises(ra.RaError):
            ra.cache8_attention(q, *ring, held)
    with pytest.raises(ra.RaError):
        ra.cache8_attention(q, *ring, W, out=q)  # aliases its input
    for k, v in ((x.half(), x), (x[:, :7], x[:, :7]), (x, x[:, :, :1]), (x.cpu(), x), (x.transpose(2, 3), x.transpose(2, 3))):
        with pytest.raises(ValueError):
            ra.cache8_append(k, v, *ring, 0)
    with pytest.raises(ra.RaError):
        ra.cache8_append(x.repeat(1, W + 1, 1, 1), x.repeat(1, W + 1, 1, 1), *ring, 0)  # two frames in a slot
    with pytest.raises(ValueError):
        ra.cache8_append(x, x, *ring, 0, k_weight=torch.ones(d + 1, device="cuda"))
    with pytest.raises(ra.RaError):
        ra.cache8_append(x, x, *ring, 0, rope=ra.rope3d(4, 3, 3, d))  # frames of 9 tokens
    with pytest.raises(ra.RaError):
        ra.cache8_append(x, x, *ring, 4, rope=ra.rope3d(4, 2, 5, d))  # frame 4 of 4
    w = torch.ones(d, device="cuda")
    for bad in (dict(q=x.float()), dict(q=x.cpu()), dict(q=x[0]), dict(k=x[:, :3]), dict(qw=w[:8]), dict(qw=w.half()),
                dict(k=None, kw=w), dict(rope=(w, w)), dict(rope=(w, w, w)), dict(q_out=torch.empty_like(x))):
        a = dict(q=x, k=x, qw=w, kw=None, rope=ra.rope3d(1, 2, 5, d), q_out=None)
        a.update(bad)
        with pytest.raises(ValueError):
            ra.qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], rope=a["rope"], q_out=a["q_out"])
    dy = torch.empty(B, H, s, d, device="cuda", dtype=torch.bfloat16)
    for args in ((x, x, dy, None), (x, None, dy, dy), (x, None, x, None)):
        with pytest.raises(ValueError):
            ra.qk_norm_rope_bwd(*args, w)
    with pytest.raises(ValueError):
        ra.qk_norm_rope_bwd(x, None, dy, None, w, workspace=torch.empty(8, device="cuda"))
    with pytest.raises(ValueError):
        ra.qk_norm_rope_bwd(x, None, dy, None, None, rope=ra.rope3d(1, 2, 5, d), dq_weight=w)
    torch.cuda.synchronize()


@pytest.mark.parametrize("nq", [1, 200])
def test_attention_without_frames(nq):
    _gpu.need_gpu()
    ring, _ = _ring(2, 2, 64, 10, 4)
    _check(torch.randn(2, 2, nq, 64, device="cuda").bfloat16(), ring, 10, 0, what="no frames")


@pytest.mark.parametrize("nq", [3, 150])
def test_every_code_at_every_scale(nq):
    """All 254 codes, in K against one-hot queries and in V under one key, at scales
    from 2^-110 to 2^110 (2^8 in K): code * scale is exact in bf16."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    for exponent in (-110, -100, -9, 0, 7, 8, 60, 110):
        k8 = torch.zeros(1, 1, 2, 128, dtype=torch.uint8)
        k8[0, 0, 0], k8[0, 0, 1] = codes[:128], codes[126:]
        k8 = k8.cuda().view(torch.float8_e4m3fn)
        unit = torch.full((1, 1, 2, 1), 2.0 ** exponent, device="cuda")
        ones = torch.ones_like(unit)
        # V: one key at a time has all the weight
        q = torch.zeros(1, 1, nq, 128, device="cuda", dtype=torch.bfloat16)
        for held, row in ((1, 0), (2, 1)):
            o = ra.cache8_attention(q, k8[:, :, row:row + 1].contiguous(), k8[:, :, row:row + 1].contiguous(),
                                    ones[:, :, :1], unit[:, :, :1].contiguous(), 1)
            want = (k8[0, 0, row].float().double() * 2.0 ** exponent).to(torch.bfloat16)
            assert torch.equal(o[0, 0], want.expand(nq, 128)), (exponent, row)
        # K: the lse of a single key is its score
        if exponent > 8:
            continue
        for at in range(0, 128, 9):
            q = torch.zeros(1, 1, nq, 128, device="cuda", dtype=torch.bfloat16)
            q[..., at] = 1
            lse = torch.empty(1, 1, nq, device="cuda")
            ra.cache8_attention(q, k8[:, :, :1].contiguous(), k8[:, :, :1].contiguous(), unit[:, :, :1].contiguous(),
                                ones[:, :, :1], 1, scale=1.0, lse=lse)
            want = float(k8[0, 0, 0, at].float().double() * 2.0 ** exponent)
            # base 2 and back: two fp32 roundings and the constants' own
            assert torch.allclose(lse.double(), torch.full_like(lse, want).double(), rtol=4 * _heads.U32, atol=1e-37)


@pytest.mark.parametrize("nq", [2, 140])
def test_non_finite_blocks_stay_where_they_are_read(nq):
    """A block whose scale is NaN poisons the batch element that attends to it, and
    nothing else: not one whose count ends before it, nor one where it lies behind
    the frames held; a NaN query poisons its own row."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 3, 2, 64, 70, 6
    (k8, v8, ks, vs), _ = _ring(B, H, d, s, W, seed=9)
    ks[0, 1, 2, 1] = float("nan")   # rows 2 * 70 + 64 ..
    vs[1, 0, 4, 0] = float("nan")   # in slot 4: not held
    vs[2, 0, 3, 0] = float("nan")   # rows 210 ..: behind the count
    q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
    q[2, 1, 1, 3] = float("nan")
    counts = torch.tensor([280, 280, 210], dtype=torch.int32, device="cuda")
    lse = torch.empty(B, H, nq, device="cuda")
    o = ra.cache8_attention(q, k8, v8, ks, vs, 4, key_counts=counts, lse=lse)
    bad = torch.isnan(o).any(-1)
    want = torch.zeros_like(bad)
    want[0, 1] = True
    want[2, 1, 1] = True
    assert torch.equal(bad, want)
    assert torch.equal(torch.isnan(lse), want)
    counts[0] = 2 * 70 + 64  # up to the block, not into it
    q[2, 1, 1, 3] = 0
    assert not bool(torch.isnan(ra.cache8_attention(q, k8, v8, ks, vs, 4, key_counts=counts)).any())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [17, 64, 128])
def test_one_tile_of_queries_over_any_number_of_steps(nq, d):
    """Up to 128 queries share a tile, and its keys are taken in two sequences of
    64-key steps that are joined at the end: none, one, and more steps in either, with
    blocks enough that the range of keys does not split."""
    _gpu.need_gpu()
    s, W = 64, 11
    counts = [64 * i + j for i in range(11) for j in (0, 1, 63)]
    ring, _ = _ring(len(counts), 5, d, s, W, seed=nq + d)
    q = torch.randn(len(counts), 5, nq, d, device="cuda").bfloat16()
    _check(q, ring, s, W, counts, what=f"{nq} queries")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [1, 80])
@pytest.mark.parametrize("down", [False, True])
def test_one_tile_of_queries_whose_maximum_moves(down, B, d):
    """Keys that grow (or shrink) by 2 ^ 1/2 from step to step: every step raises its
    sequence's maximum, or adds next to nothing to it."""
    _gpu.need_gpu()
    s, W = 64, 11
    (k8, v8, ks, vs), _ = _ring(B, 2, d, s, W, seed=d + B)
    ramp = 2.0 ** (torch.arange(W, device="cuda").float() / 2)
    ks.mul_((ramp.flip(0) if down else ramp)[None, None, :, None])
    q = torch.randn(B, 2, 100, d, device="cuda").bfloat16()
    # Every second scale is no power of two: the kernel rounds it, and code * scale, to
    # bf16 (two roundings, each at most BF16 of the value).  The keys so rounded are bf16
    # operands whose products are exact again, as _reference's bounds want them.
    ra = _gpu.ra()
    lse = torch.empty(B, 2, 100, device="cuda")
    o = ra.cache8_attention(q, k8, v8, ks, vs, W, lse=lse)
    true = _values(k8, ks, s)
    keys = _values(k8, ks.bfloat16(), s).bfloat16()
    assert bool(((keys.double() - true).abs() <= true.abs() * (2 * _heads.BF16 + _heads.BF16 ** 2)).all())
    want, want_lse, ob, lb = _reference(q, keys, v8, torch.ones_like(ks), vs, s, [W * s] * B, 1 / math.sqrt(d))
    off = ((o.double().cpu() - want).abs() / ob).max().item()
    assert off <= 1, f"o off by {off:.3g} of the bound"
    off = ((lse.double().cpu() - want_lse).abs() / lb).max().item()
    assert off <= 1, f"lse off by {off:.3g} of the bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,nq,s", [(4, 37, 200, 60), (2, 3, 300, 60), (4, 37, 129, 60), (2, 74, 257, 130), (1, 2, 513, 200)])
def test_one_and_two_tiles_of_queries_a_block(B, H, nq, s, d):
    """Heads enough to fill the SMs with blocks of two tiles, or few, with tiles of a few
    rows at the end."""
    _gpu.need_gpu()
    W = 10
    counts = [s * W - 7 * b for b in range(B)]
    ring, _ = _ring(B, H, d, s, W, seed=nq)
    q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
    _check(q, ring, s, W, counts, what=f"{nq} queries")


def test_non_finite_blocks_of_one_tile_of_queries():
    test_non_finite_blocks_stay_where_they_are_read(70)


@pytest.mark.parametrize("nq", [1, 33, 260])
def test_same_bits_on_any_stream_and_in_a_graph(nq):
    """Two runs, a run on another stream, and a captured graph replayed after the ring
    and the counts changed, agree bit for bit with plain calls; two graphs with
    workspaces of their own may be replayed in turn."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W, held = 2, 3, 128, 50, 60, 55
    ring, _ = _ring(B, H, d, s, W, seed=2)
    other, _ = _ring(B, H, d, s, W, seed=3)
    q = torch.randn(B, H, nq, d, device="cuda").bfloat16()
    counts = torch.tensor([2750, 1333], dtype=torch.int32, device="cuda")
    call = lambda **kw: ra.cache8_attention(q, *ring, held, key_counts=counts, **kw)  # noqa: E731
    first = call()
    assert torch.equal(first, call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = call(stream=side)
    side.synchronize()
    assert torch.equal(first, there)
    graphs, held_out = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            held_out.append(call())
    for t, o in zip(ring, other):
        t.view(torch.uint8).copy_(o.view(torch.uint8))
    counts.copy_(torch.tensor([77, 2749], dtype=torch.int32))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    again = call()
    assert not torch.equal(first, again)
    assert all(torch.equal(o, again) for o in held_out)


# -------------------------------------------------------------- the class, in a run
@pytest.mark.parametrize("B,H,d,grid,W,f", [(1, 2, 64, (1, 1), 40, 90), (1, 2, 128, (5, 26), 3, 8),
                                           (2, 1, 64, (8, 12), 2, 5)], ids=lambda x: str(x))
def test_stream(B, H, d, grid, W, f):
    """Frames streamed through SwcCache8 as a model would (raw projections; norm,
    rotation, append, attention): every frame's output against attention in fp64 over
    the last W frames of normed and rotated keys, the quantisation included."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    s = grid[0] * grid[1]
    n = f * s
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = torch.randn(B, n, 3 * H, d, generator=g, device="cuda").bfloat16().split(H, dim=2)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = ra.rope3d(f, *grid, d)
    cache = ra.SwcCache8(B, H, d, s, W)
    for i in range(f):
        at = slice(i * s, (i + 1) * s)
        lse = torch.empty(B, H, s, device="cuda")
        o = cache.step(q[:, at], k[:, at], v[:, at], wq, wk, rope, EPS, lse=lse)
        assert cache.info == dict(frames_seen=i + 1, frames_held=min(i + 1, W))
        yq, _ = ra.qk_norm_rope(q[:, at], None, wq, rope=rope, frame0=i, eps=EPS)
        want, want_lse, ob, lb = _reference(yq, *(t[:, :, :min(i + 1, W) * s] for t in (cache.k8, cache.v8)),
                                            *(t[:, :, :min(i + 1, W)] for t in (cache.k_scale, cache.v_scale)), s,
                                            [min(i + 1, W) * s] * B, 1 / math.sqrt(d))
        assert bool(((o.double().cpu() - want).abs() <= ob).all()) and bool(((lse.double().cpu() - want_lse).abs() <= lb).all())
        # against unquantised keys and values: an e4m3 rounding is off by at most 2^-4 of a value; over d channels
        # and the keys it averages, so that the whole stays within 2^-4 of the output's norm
        first = max(0, i - W + 1) * s
        k64, _ = _heads.norm_rope(k[:, first:(i + 1) * s], wk, rope, max(0, i - W + 1), EPS)
        v64 = v[:, first:(i + 1) * s].double().cpu().transpose(1, 2)
        plain = torch.softmax(yq.double().cpu() @ k64.transpose(2, 3) / math.sqrt(d), -1) @ v64
        assert (o.double().cpu() - plain).norm() <= 2.0 ** -4 * plain.norm()
    assert ra.device_status() == ra.RA_OK


def test_many_frames_at_once_and_reset():
    """Appending frames one by one or all at once fills the ring alike (more than W
    frames too), also without norm or rotation; reset forgets them."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 2, 64, 90, 4
    k, v = (torch.randn(B, 7 * s, H, d, device="cuda").bfloat16() for _ in range(2))
    one, all_ = ra.SwcCache8(B, H, d, s, W), ra.SwcCache8(B, H, d, s, W)
    for i in range(7):
        one.append(k[:, i * s:(i + 1) * s], v[:, i * s:(i + 1) * s])
    all_.append(k, v)
    assert one.info == all_.info == dict(frames_seen=7, frames_held=4)
    for a, b in zip(one._ring, all_._ring):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q = torch.randn(B, s, H, d, device="cuda").bfloat16()
    a, b = one.step(q, k[:, :s], v[:, :s]), all_.step(q, k[:, :s], v[:, :s])
    assert torch.equal(a, b)
    one.reset()
    assert one.info == dict(frames_seen=0, frames_held=0)
    assert bool((one.attend(q.transpose(1, 2).contiguous()) == 0).all())
    one.append(k[:, :s], v[:, :s])
    assert one.frames_held == 1


def test_captured_steps_are_refused():
    """A step's frame number is host state: capturing it is refused, the functions
    under it are not, and the cache is as it was."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    cache = ra.SwcCache8(1, 1, 64, 8, 2)
    x = torch.randn(1, 8, 1, 64, device="cuda").bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError):
            cache.step(x, x, x)
        with pytest.raises(RuntimeError):
            cache.append(x, x)
        ra.cache8_append(x, x, *cache._ring, 0)
        o = ra.cache8_attention(x.transpose(1, 2).contiguous(), *cache._ring, 1)
    assert cache.info == dict(frames_seen=0, frames_held=0)
    graph.replay()
    torch.cuda.synchronize()
    want = cache.step(x, x, x)
    assert torch.equal(o, want)


def test_offsets_beyond_32_bits():
    """A ring of 4.4e9 codes: the last head's rows are written, read and attended to."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, d, s, W = 1, 35, 128, 1000, 1000
    k8 = torch.zeros(B, H, s * W, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v8 = torch.zeros_like(k8.view(torch.uint8)).view(torch.float8_e4m3fn)
    ks, vs = (torch.ones(B, H, W, 16, device="cuda") for _ in range(2))
    k, v = (torch.randn(B, s, H, d, device="cuda").bfloat16() for _ in range(2))
    ra.cache8_append(k, v, k8, v8, ks, vs, W - 1)
    small, _ = _ring(B, H, d, s, 1)
    ra.cache8_append(k, v, *small, 0)
    assert torch.equal(k8[:, :, -s:].view(torch.uint8), small[0].view(torch.uint8))
    assert torch.equal(vs[:, :, -1], small[3][:, :, 0])
    assert int(k8.view(torch.uint8)[:, :, :-s].count_nonzero()) == 0
    # zeros score 0: with q along a key, that key's weight is e^x / (e^x + 10^6 - 1 + ..)
    for nq in (1, 130):
        q = torch.zeros(B, H, nq, d, device="cuda").bfloat16()
        q += k[:, -1, :, None, :] * 6
        o = ra.cache8_attention(q, k8, v8, ks, vs, W)
        values, keys = _values(small[1], small[3], s), _values(small[0], small[2], s)
        x = q.double().cpu() @ keys.transpose(2, 3) / math.sqrt(d)
        top = x.amax(-1, keepdim=True).clamp(min=0)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True) + (W - 1) * s * torch.exp(-top)
        want = p @ values / total
        # P's and o's roundings, and fp32 sums over 10^6 keys kept in at most 2^14 partial additions each
        bound = want.abs() * _heads.BF16 + (p @ values.abs() / total) * (_heads.BF16 + 2.0 ** -9)
        assert bool(((o.double().cpu() - want).abs() <= bound).all())
