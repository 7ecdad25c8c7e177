"""Per-head norm and 3-axis rotation of Q and K, and their gradient, against the
64-bit forms of tests/_heads.py on the same inputs, element by element within the
bounds that the roundings give."""
import pytest
import torch

from tests import _gpu, _heads

pytestmark = pytest.mark.gpu

EPS = 1e-6
#        B, f, gh, gw, Hq, Hk, d,   axes (None: the default split)
SHAPES = [
    (1, 1, 1, 1, 1, 1, 64, None),          # one token, one head
    (1, 1, 1, 1, 40, 40, 128, None),
    (2, 3, 5, 7, 3, 3, 128, None),         # odd grid
    (1, 2, 9, 11, 5, 2, 64, None),         # fewer heads of k
    (3, 1, 16, 16, 12, 12, 64, (16, 24, 24)),
    (1, 4, 3, 50, 9, 9, 128, (0, 64, 64)),  # an image model: no time axis
    (1, 33, 1, 1, 17, 17, 128, (128, 0, 0)),  # text-like: time alone
    (1, 2, 6, 13, 4, 4, 128, (16, 40, 42)),  # 30 channels are not rotated
    (2, 5, 13, 17, 8, 8, 128, (2, 62, 64)),
]


def _inputs(shape, seed, packed, w32):
    B, f, gh, gw, Hq, Hk, d, axes = shape
    n = f * gh * gw
    g = torch.Generator(device="cuda").manual_seed(seed)
    if packed:
        x = torch.randn(B, n, Hq + 2 * Hk, d, generator=g, device="cuda").bfloat16()
        q, k, _ = x.split([Hq, Hk, Hk], dim=2)
    else:  # head-major storage of a token-major view
        q = torch.randn(B, Hq, n, d, generator=g, device="cuda").bfloat16().transpose(1, 2)
        k = torch.randn(B, Hk, n, d, generator=g, device="cuda").mul(30).bfloat16().transpose(1, 2)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    w = w if w32 else [x.bfloat16() for x in w]
    dq = torch.randn(B, Hq, n, d, generator=g, device="cuda").bfloat16()
    dk = torch.randn(B, Hk, n, d, generator=g, device="cuda").mul(1e-3).bfloat16()
    return q, k, w, dq, dk


def _within(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    worst = (off / bound).max().item()
    assert bool((off <= bound).all()), f"{what}: off by {worst:.3g} of the bound"


@pytest.mark.parametrize("norm,rotated", [(True, True), (True, False), (False, True)],
                         ids=["norm+rope", "norm", "rope"])
@pytest.mark.parametrize("packed,w32", [(True, False), (False, True)], ids=["packed-bf16w", "headmajor-fp32w"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:7])))
def test_forward_and_backward(shape, packed, w32, norm, rotated):
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, f, gh, gw, Hq, Hk, d, axes = shape
    n, frame0 = f * gh * gw, 5
    q, k, w, dq_out, dk_out = _inputs(shape, 100 + n + Hq, packed, w32)
    wq, wk = w if norm else (None, None)
    rope = ra.rope3d(frame0 + f, gh, gw, d, axes=axes) if rotated else None
    gq, gk = _gpu.Guarded((B, Hq, n, d), torch.bfloat16), _gpu.Guarded((B, Hk, n, d), torch.bfloat16)
    yq, yk = ra.qk_norm_rope(q, k, wq, wk, rope=rope, frame0=frame0, eps=EPS, q_out=gq.t, k_out=gk.t)
    _gpu.check_canaries(gq, gk, what="norm + rope")
    for name, x, weight, y in (("q", q, wq, yq), ("k", k, wk, yk)):
        _within(y, *_heads.norm_rope(x, weight, rope, frame0, EPS), f"{name} forward")
    hq, hk = _gpu.Guarded((B, n, Hq, d), torch.bfloat16), _gpu.Guarded((B, n, Hk, d), torch.bfloat16)
    ws = _gpu.Guarded((max(4, ra.ra_qk_norm_rope_bwd_workspace_bytes(d) // 4),), torch.float32)
    gw_q, gw_k = _gpu.Guarded((d,), torch.float32), _gpu.Guarded((d,), torch.float32)
    got = ra.qk_norm_rope_bwd(q, k, dq_out, dk_out, wq, wk, rope=rope, frame0=frame0, eps=EPS, dq=hq.t, dk=hk.t,
                              dq_weight=gw_q.t if norm else None, dk_weight=gw_k.t if norm else None, workspace=ws.t)
    _gpu.check_canaries(hq, hk, ws, gw_q, gw_k, what="norm + rope backward")
    for name, x, dy, weight, dx, dw in (("q", q, dq_out, wq, got[0], got[2]), ("k", k, dk_out, wk, got[1], got[3])):
        dx64, dx_bound, dw64, dw_bound = _heads.norm_rope_bwd(x, dy, weight, rope, frame0, EPS)
        _within(dx, dx64, dx_bound, f"d{name}")
        if norm:
            _within(dw, dw64, dw_bound, f"d{name} weight")
        else:
            assert dw is None


def test_gradient_against_differences():
    """<dx, v> against the central difference of <y, dy> along v, in 64 bits: the
    formula behind the bounds is the forward's gradient."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    shape = (2, 3, 4, 5, 3, 2, 64, None)
    q, k, w, dq_out, dk_out = _inputs(shape, 7, True, True)
    rope = ra.rope3d(4, 4, 5, 64)
    got = ra.qk_norm_rope_bwd(q, k, dq_out, dk_out, *w, rope=rope, frame0=1, eps=EPS)
    for x, dy, weight, dx, dw in ((q, dq_out, w[0], got[0], got[2]), (k, dk_out, w[1], got[1], got[3])):
        x64, w64, dy64 = x.double().cpu(), weight.double().cpu(), dy.double().cpu()
        g = torch.Generator().manual_seed(3)
        v, u = torch.randn(x64.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64)
        loss = lambda a, b: (_heads.norm_rope(a, b, rope, 1, EPS)[0] * dy64).sum()  # noqa: E731
        step = 1e-5
        want = (loss(x64 + step * v, w64 + step * u) - loss(x64 - step * v, w64 - step * u)) / (2 * step)
        _, bound, _, dw_bound = _heads.norm_rope_bwd(x, dy, weight, rope, 1, EPS)
        have = (dx.double().cpu() * v).sum() + (dw.double().cpu() * u).sum()
        # the difference's own error: step^2 / 6 of the third derivative (of order 10 * |dy| sums here)
        slack = (bound * v.abs()).sum() + (dw_bound * u.abs()).sum() + 1e-8 * dy64.abs().sum()
        assert abs(have - want) <= slack, (float(have), float(want), float(slack))


def test_tables_and_far_positions():
    """The tables hold cos and sin to half an fp32 step (plus the 64-bit angle's own
    error), at frame 10^6 too; a call far into a stream uses those rows."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    rope = ra.rope3d(1_000_001, 3, 2, 64, axes=(24, 20, 20), base=5000.0)
    want = _heads.table64(1001, 12, 5000.0, start=999_000)
    assert (rope.t[999_000:1_000_001].double().cpu() - want).abs().max() <= 2.0 ** -25 + 1e-9
    assert (rope.h.double().cpu() - _heads.table64(3, 10, 5000.0)).abs().max() <= 2.0 ** -25 + 1e-9
    x = torch.randn(1, 6, 2, 64, device="cuda").bfloat16()
    y, none = ra.qk_norm_rope(x, rope=rope, frame0=1_000_000)
    assert none is None
    _within(y, *_heads.norm_rope(x, None, rope, 1_000_000, EPS), "far frame")


def test_values_that_are_not_ordinary():
    """Zero rows stay zero (their gradient is dy * w / sqrt(eps)); a NaN or an
    infinity stays in its own row; large and tiny rows keep the formula."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    x = torch.randn(1, 6, 2, 64, device="cuda").bfloat16()
    x[0, 1] = 0
    x[0, 2, 0, 5] = float("nan")
    x[0, 3, 1, 9] = float("inf")
    x[0, 4] *= 1e15
    x[0, 5] *= 1e-15
    w = torch.ones(64, device="cuda")
    y, _ = ra.qk_norm_rope(x, None, w)
    y64, bound = _heads.norm_rope(x, w, None, 0, EPS)
    ok = torch.ones(2, 6, dtype=torch.bool)
    ok[0, 2] = ok[1, 3] = False
    got = y.double().cpu()[0]
    assert bool(((got - y64[0]).abs() <= bound[0])[ok].all())
    assert bool(torch.isnan(got[0, 2]).all()) and bool(torch.isnan(got[1, 3]).any())
    dy = torch.randn(1, 2, 6, 64, device="cuda").bfloat16()
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    dx, _, dw, _ = ra.qk_norm_rope_bwd(clean, None, dy, None, w)
    dx64, dx_bound, dw64, dw_bound = _heads.norm_rope_bwd(clean, dy, w, None, 0, EPS)
    _within(dx, dx64, dx_bound, "dx")
    _within(dw, dw64, dw_bound, "dw")


def test_no_tokens():
    _gpu.need_gpu()
    ra = _gpu.ra()
    x, w = torch.empty(2, 0, 3, 64, device="cuda", dtype=torch.bfloat16), torch.ones(64, device="cuda")
    y, k = ra.qk_norm_rope(x, x, w, w)
    assert y.shape == k.shape == (2, 3, 0, 64)
    dw = torch.full((64,), 3.0, device="cuda")
    dx, _, dw, _ = ra.qk_norm_rope_bwd(x, None, y, None, w, dq_weight=dw)
    assert dx.shape == x.shape and bool((dw == 0).all())


def test_broadcast_input_and_packed_gradient():
    """An expanded input is read with stride 0; dq and dk are written into slots of
    one packed gradient and nothing else of it is touched."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    one = torch.randn(1, 20, 1, 128, device="cuda").bfloat16()
    q = one.expand(2, 20, 3, 128)
    w = torch.randn(128, device="cuda")
    y, _ = ra.qk_norm_rope(q, None, w)
    _within(y, *_heads.norm_rope(q, w, None, 0, EPS), "expanded")
    packed = torch.full((2, 20, 3 + 2 + 2, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    dq, dk, rest = packed.split([3, 2, 2], dim=2)
    k = torch.randn(2, 20, 2, 128, device="cuda").bfloat16()
    dyq, dyk = torch.randn(2, 3, 20, 128, device="cuda").bfloat16(), torch.randn(2, 2, 20, 128, device="cuda").bfloat16()
    rope = ra.rope3d(1, 4, 5, 128)
    ra.qk_norm_rope_bwd(q, k, dyq, dyk, w, w, rope=rope, dq=dq, dk=dk)
    _within(dq, *_heads.norm_rope_bwd(q, dyq, w, rope, 0, EPS)[:2], "packed dq")
    _within(dk, *_heads.norm_rope_bwd(k, dyk, w, rope, 0, EPS)[:2], "packed dk")
    assert bool((rest == 7.0).all())
    # and with q, k and v side by side in each head: [B, n, H, 3, d]
    packed = torch.full((2, 20, 2, 3, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    dyq = dyk.flip(2).contiguous()
    ra.qk_norm_rope_bwd(k, k, dyq, dyk, w, w, rope=rope, dq=packed[:, :, :, 0], dk=packed[:, :, :, 1])
    _within(packed[:, :, :, 0], *_heads.norm_rope_bwd(k, dyq, w, rope, 0, EPS)[:2], "dq beside dk")
    _within(packed[:, :, :, 1], *_heads.norm_rope_bwd(k, dyk, w, rope, 0, EPS)[:2], "dk beside dq")
    assert bool((packed[:, :, :, 2] == 7.0).all())


def test_same_bits_every_time_on_any_stream_and_in_a_graph():
    """Two runs agree bit for bit (the weights' gradients too); so do a run on
    another stream and a captured graph replayed on new inputs."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    shape = (2, 7, 11, 13, 9, 9, 128, None)
    q, k, w, dq_out, dk_out = _inputs(shape, 11, True, False)
    rope = ra.rope3d(7, 11, 13, 128)

    def both(stream=None):
        return (*ra.qk_norm_rope(q, k, *w, rope=rope, stream=stream),
                *ra.qk_norm_rope_bwd(q, k, dq_out, dk_out, *w, rope=rope, stream=stream))

    first = both()
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    q.mul_(-2)
    dk_out.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    again = both()
    assert all(torch.equal(a, b) for a, b in zip(held, again))
    assert not torch.equal(first[0], again[0])


def test_norm_and_rotation_around_the_attention(orc):
    """The operators as a training step runs them: q and k normed and rotated, radial
    attention forward and backward, and back through the rotation and the norm --
    against autograd of the whole chain in fp64 (attention restricted to the mask's
    kept pairs).  Bars: the attention's own (relative 5e-3 forward and backward)
    widened by the two more bf16 roundings on the way (of q, k and of dq, dk, each
    at most BF16 = 2^-8 a value, averaging out to under 2^-9 over a tensor)."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    f, gh, gw, H, d = 4, 8, 10, 2, 64
    s, n = gh * gw, f * gh * gw
    shape = (1, f, gh, gw, H, H, d, None)
    q, k, w, _, _ = _inputs(shape, 23, True, True)
    g = torch.Generator(device="cuda").manual_seed(5)
    v, do = (torch.randn(1, H, n, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    rope = ra.rope3d(f, gh, gw, d)
    mask = ra.Mask("radial", f, s)
    yq, yk = ra.qk_norm_rope(q, k, *w, rope=rope, eps=EPS)
    lse = torch.empty(1, H, n, device="cuda")
    o = ra.attention_fwd(yq, yk, v, mask, mode="token_exact", lse=lse)
    dyq, dyk, dv = ra.attention_bwd(yq, yk, v, o, do, lse, mask, mode="token_exact")
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, dyq, dyk, *w, rope=rope, eps=EPS)
    assert ra.device_status() == ra.RA_OK

    i = torch.arange(n)
    fr, pos = i // s, i % s
    dist = (fr[:, None] - fr[None, :]).abs().clamp(min=1)
    band = 2 ** torch.floor(torch.log2(dist.double())).long()
    kept = ((pos[:, None] - pos[None, :]).abs() + 1) * band <= s  # eq. 4; f <= s, so every band has width >= 1
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v, *w)]
    q64 = _heads.norm_rope(leaves[0].detach(), w[0], rope, 0, EPS)[0]
    assert q64.shape == yq.shape

    def chain(x, weight):
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
        return _heads.rotate(x, *_heads.angles(rope, 0, n, d)).transpose(1, 2)

    score = chain(leaves[0], leaves[3]) @ chain(leaves[1], leaves[4]).transpose(2, 3) / d ** 0.5
    out = torch.softmax(score.masked_fill(~kept, float("-inf")), -1) @ leaves[2]
    out.backward(do.double().cpu())
    for name, got, want in (("o", o, out), ("dq", dq, leaves[0].grad), ("dk", dk, leaves[1].grad),
                            ("dv", dv, leaves[2].grad), ("dwq", dwq, leaves[3].grad), ("dwk", dwk, leaves[4].grad)):
        got, want = got.double().cpu(), want.detach()
        rel = float((got - want).norm() / want.norm())
        assert rel <= 5e-3 + 2 * 2.0 ** -9, f"{name}: {rel:.3e}"
