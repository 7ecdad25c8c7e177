"""What is measured of the operators around the attention kernels: the per-head
norm and three-axis rotation of Q and K (forward and backward), the append of
new frames to an 8-bit key/value ring, and attention over that ring.

A case names one operator ("op") and its sizes:
  norm_rope      q, k [B, n, H, d] -> normed, rotated q, k [B, H, n, d]
  norm_rope_bwd  its gradients: dq, dk [B, n, H, d] and those of the norm weights
  append         k, v of `frames` new frames into the e4m3 ring of W frames
  attend         nq queries per head over the first `held` frames of the ring
"""
import math

import torch

own = False

BLOCK = 64       # tokens of one frame that share a scale in the 8-bit ring
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------- the cases
def _nr(name, op, B, f, gh, gw, H, d, packed=True, norm=True, rope=True, w32=False, frame0=0, Hk=0):
    return dict(name=name, op=op, B=B, f=f, gh=gh, gw=gw, H=H, Hk=Hk or H, d=d, packed=packed, norm=norm, rope=rope,
                w32=w32, frame0=frame0)


def _ap(name, B, frames, gh, gw, H, d, W, frame, norm=True, rope=True, packed=True, w32=False):
    return dict(name=name, op="append", B=B, frames=frames, gh=gh, gw=gw, H=H, d=d, W=W, frame=frame, norm=norm,
                rope=rope, packed=packed, w32=w32)


def _at(name, B, H, d, s, W, held, nq, ragged=False):
    return dict(name=name, op="attend", B=B, H=H, d=d, s=s, W=W, held=held, nq=nq, ragged=ragged)


def listed():
    return [
        # the smallest call: a short clip of small frames, one head; launch latency counts
        _nr("norm_rope_tiny", "norm_rope", 1, 8, 8, 8, 1, 64),
        # a batch of short clips, rotation only (a model without norms of Q and K)
        _nr("norm_rope_batch_rope_only", "norm_rope", 2, 16, 16, 16, 12, 64, norm=False),
        # a whole video of 108000 tokens out of the fused QKV projection
        _nr("norm_rope_108k", "norm_rope", 1, 30, 45, 80, 24, 128),
        # training on one odd-sized frame (fp32 norm weights kept by the optimiser)
        _nr("norm_rope_bwd_frame", "norm_rope_bwd", 1, 1, 31, 51, 40, 128, w32=True, frame0=7),
        # training on a whole video of 63960 tokens
        _nr("norm_rope_bwd_64k", "norm_rope_bwd", 1, 41, 30, 52, 40, 128),
        # serving single tokens: eight streams, one token each, scale per token
        _ap("append_tokens", 8, 1, 1, 1, 24, 128, 4096, 70001),
        # streaming: one frame of 1560 tokens replaces the oldest of 16
        _ap("append_frame", 1, 1, 30, 52, 40, 128, 16, 37),
        # the window filled at once from a given video; odd frames, so blocks end early
        _ap("append_window", 1, 12, 45, 79, 24, 128, 16, 9),
        # the smallest call: one query over a few hundred keys
        _at("attend_tiny", 1, 12, 64, 37, 8, 7, 1),
        # serving single tokens: eight streams of unequal length, long caches
        _at("attend_tokens_32k", 8, 24, 128, 1, 32768, 32768, 1, ragged=True),
        # streaming small frames in a batch, the window not yet full
        _at("attend_small_frames", 2, 12, 64, 256, 16, 11, 256),
        # streaming: the queries of one 1560-token frame over the full window
        _at("attend_frame", 1, 40, 128, 1560, 16, 16, 1560),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attend"])
    d = rng.choice([64, 128])
    if op in ("norm_rope", "norm_rope_bwd"):
        gh, gw, H, B = _log(rng, 1, 45), _log(rng, 1, 80), rng.randint(1, 40), rng.choice([1, 1, 2, 3])
        most = 320_000_000 if op == "norm_rope" else 300_000_000  # the largest listed: 332e6 and 327e6 values a tensor
        f = _log(rng, 1, max(1, min(128, most // (B * gh * gw * H * d))))
        norm = rng.random() < 0.8
        return dict(op=op, B=B, f=f, gh=gh, gw=gw, H=H, Hk=rng.choice([H, H, max(1, H // 2)]), d=d,
                    packed=rng.random() < 0.6, norm=norm, rope=not norm or rng.random() < 0.8,
                    w32=rng.random() < 0.5, frame0=rng.choice([0, rng.randint(1, 500)]))
    if op == "append":
        gh, gw, H, B = _log(rng, 1, 45), _log(rng, 1, 80), rng.randint(1, 40), rng.choice([1, 1, 2, 8])
        W = _log(rng, 1, max(1, min(64, 150_000_000 // (B * gh * gw * H * d))))
        return dict(op=op, B=B, frames=rng.choice([1, rng.randint(1, W)]), gh=gh, gw=gw, H=H, d=d, W=W,
                    frame=rng.choice([0, rng.randint(0, 3000)]), norm=rng.random() < 0.8, rope=rng.random() < 0.8,
                    packed=rng.random() < 0.7, w32=rng.random() < 0.5)
    if rng.random() < 0.5:  # few queries over a long cache
        nq, B, H = rng.choice([1, 1, rng.randint(2, 40)]), rng.choice([1, 2, 4, 8]), rng.randint(1, 40)
        s = rng.choice([1, 1, _log(rng, 2, 600)])
        W = max(1, _log(rng, 64, max(65, min(200_000, 700_000_000 // (B * H * d)))) // s)
    else:  # the queries of a frame over the window
        nq = _log(rng, 41, 3600)
        s, B, H = rng.choice([nq, _log(rng, 30, 3600)]), rng.choice([1, 1, 2]), rng.randint(1, 40)
        rows = min(60_000, 1_400_000_000 // (B * H * nq), 150_000_000 // (B * H * d))
        W = max(1, _log(rng, s, max(s + 1, rows)) // s)
    held = rng.choice([W, rng.randint(1, W)])
    return dict(op="attend", B=B, H=H, d=d, s=s, W=W, held=held, nq=nq, ragged=B > 1 and rng.random() < 0.5)


def axes_of(d):
    """Channels of the time, height and width axes: height and width get 2 * (d // 6) each, time the rest."""
    return d - 4 * (d // 6), 2 * (d // 6), 2 * (d // 6)


def counts_of(case):
    """Keys that each batch element attends to."""
    n, B = case["held"] * case["s"], case["B"]
    return [n * (b + 1) // B for b in range(B)] if case["ragged"] else [n] * B


# ------------------------------------------------------------------ the inputs
def _table(start, length, dim):
    """fp32 [length, dim / 2, 2]: cos and sin of position * BASE^(-2 i / dim), the angle in 64 bits."""
    pos = torch.arange(start, start + length, device="cuda", dtype=torch.float64)
    i = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    a = pos[:, None] * torch.pow(torch.tensor(BASE, dtype=torch.float64, device="cuda"), -2.0 * i / dim)
    return torch.stack([a.cos(), a.sin()], -1).float()


def _heads(g, B, n, H, d, gain=1.0):
    x = torch.randn(B, n, H, d, generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(gain) if gain != 1.0 else x


def _packed(g, B, n, heads, d):
    """Views of one projection's output [B, n, sum(heads) * d]: what a fused QKV product gives."""
    x = torch.randn(B, n, sum(heads), d, generator=g, device="cuda", dtype=torch.bfloat16)
    return list(x.split(heads, dim=2))


def _weight(g, d, w32):
    w = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
    return w if w32 else w.bfloat16()


def _scales(amax):
    """The power of two that brings a block's largest value to at most 448."""
    m, e = torch.frexp(amax)
    k = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), k), torch.ones_like(amax))


def _per_token(scale, s):
    """[..., frames, blocks] -> [..., frames * s, 1]"""
    x = scale.repeat_interleave(min(BLOCK, s), dim=-1)[..., :s]
    return x.reshape(*scale.shape[:-2], -1, 1)


def _quantise(x, s):
    """x fp32 [B, H, frames * s, d] -> e4m3 codes of the same shape and scales [B, H, frames, blocks]."""
    B, H, n, d = x.shape
    size = min(BLOCK, s)
    blocks = -(-s // size)
    y = torch.nn.functional.pad(x.view(B, H, n // s, s, d), (0, 0, 0, blocks * size - s))
    scale = _scales(y.abs().reshape(B, H, n // s, blocks, size * d).amax(-1))
    return (x / _per_token(scale, s)).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    B, H, d = c["B"], c["H"], c["d"]
    if c["op"] == "attend":
        rows = c["W"] * c["s"]
        k = torch.randn(B, H, rows, d, generator=g, device="cuda")
        k8, k_scale = _quantise(k, c["s"])
        k.normal_(generator=g)
        v8, v_scale = _quantise(k.mul_(3.0), c["s"])
        q = torch.randn(B, H, c["nq"], d, generator=g, device="cuda", dtype=torch.bfloat16)
        counts = torch.tensor(counts_of(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
        return dict(case=c, q=q, k8=k8, v8=v8, k_scale=k_scale, v_scale=v_scale, counts=counts)
    s = c["gh"] * c["gw"]
    frames = c["frames"] if c["op"] == "append" else c["f"]
    first = c["frame"] if c["op"] == "append" else c["frame0"]
    n = frames * s
    t, h, w = axes_of(d)
    # the tables that a user's program keeps: the time axis from frame 0 on
    rope = (_table(0, first + frames, t), _table(0, c["gh"], h), _table(0, c["gw"], w)) if c["rope"] else None
    state = dict(case=c, rope=rope, first=first)
    if c["op"] == "append":
        if c["packed"]:
            _, state["k"], state["v"] = _packed(g, B, n, [H, H, H], d)
        else:
            state["k"], state["v"] = _heads(g, B, n, H, d), _heads(g, B, n, H, d, 4.0)
        state["kw"] = _weight(g, d, c["w32"]) if c["norm"] else None
        blocks, W = -(-s // BLOCK), c["W"]
        # a ring that holds earlier frames
        code = torch.randint(0, 120, (B, H, W * s, d), generator=g, device="cuda", dtype=torch.uint8)
        state["k8"] = code.view(torch.float8_e4m3fn)
        state["v8"] = code.flip(1).contiguous().view(torch.float8_e4m3fn)
        state["k_scale"] = torch.full((B, H, W, blocks), 2.0 ** -6, device="cuda")
        state["v_scale"] = torch.full((B, H, W, blocks), 2.0 ** -7, device="cuda")
        return state
    if c["packed"]:
        state["q"], state["k"], _ = _packed(g, B, n, [H, c["Hk"], c["Hk"]], d)
    else:
        state["q"], state["k"] = _heads(g, B, n, H, d, 2.0), _heads(g, B, n, c["Hk"], d, 0.5)
    state["qw"] = _weight(g, d, c["w32"]) if c["norm"] else None
    state["kw"] = _weight(g, d, c["w32"]) if c["norm"] else None
    if c["op"] == "norm_rope_bwd":  # attention's gradients, small as behind a mean over many tokens
        state["dq"] = torch.randn(B, H, n, d, generator=g, device="cuda", dtype=torch.bfloat16).mul_(2.0 ** -10)
        state["dk"] = torch.randn(B, c["Hk"], n, d, generator=g, device="cuda", dtype=torch.bfloat16).mul_(2.0 ** -10)
    return state


# -------------------------------------------------------------- the plain forms
def _angles(rope, first, n, gh, gw):
    """cos and sin [n, 1, d / 2] of the tokens of frames first, first + 1, ..."""
    i = torch.arange(n, device="cuda")
    at = torch.cat([rope[0][first + i // (gh * gw)], rope[1][i // gw % gh], rope[2][i % gw]], dim=1)
    return at[:, None, :, 0], at[:, None, :, 1]


def _rotate(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _norm_rope(x, w, rope, first, gh, gw):
    """fp32 [B, n, H, d]"""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(x, *_angles(rope, first, x.shape[1], gh, gw)) if rope is not None else x


def _norm_rope_bwd(x, dy, w, rope, first, gh, gw):
    """dx bf16 [B, n, H, d] and the weight's gradient fp32 [d] (None without a norm)."""
    a = dy.transpose(1, 2).float()
    if rope is not None:
        cos, sin = _angles(rope, first, a.shape[1], gh, gw)
        a = _rotate(a, cos, -sin)
    if w is None:
        return a.bfloat16(), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * r
    dw = (a * x).sum((0, 1, 2))
    a = a * w.float()
    return (r * (a - x * (a * x).mean(-1, keepdim=True))).bfloat16(), dw


def _run_plain(t):
    c = t["case"]
    if c["op"] == "attend":
        n, scale = c["held"] * c["s"], 1.0 / math.sqrt(c["d"])
        k = t["k8"][:, :, :n].float() * _per_token(t["k_scale"], c["s"])[:, :, :n]
        s = torch.matmul(t["q"].float(), k.transpose(2, 3)) * scale
        del k
        if t["counts"] is not None:
            out = torch.arange(n, device="cuda") >= t["counts"][:, None]
            s = s.masked_fill_(out[:, None, None, :], -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-3e38)
        p = s.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        v = t["v8"][:, :, :n].float() * _per_token(t["v_scale"], c["s"])[:, :, :n]
        o = torch.matmul(p, v) / l.clamp(min=1e-37)
        return o.bfloat16(), (m + l.log()).squeeze(-1)
    gh, gw, first, rope = c["gh"], c["gw"], t["first"], t["rope"]
    if c["op"] == "norm_rope":
        return (_norm_rope(t["q"], t["qw"], rope, first, gh, gw).bfloat16().transpose(1, 2).contiguous(),
                _norm_rope(t["k"], t["kw"], rope, first, gh, gw).bfloat16().transpose(1, 2).contiguous())
    if c["op"] == "norm_rope_bwd":
        dq, dqw = _norm_rope_bwd(t["q"], t["dq"], t["qw"], rope, first, gh, gw)
        dk, dkw = _norm_rope_bwd(t["k"], t["dk"], t["kw"], rope, first, gh, gw)
        return dq, dk, dqw, dkw
    s, W = gh * gw, c["W"]
    slots = (first + torch.arange(c["frames"], device="cuda")) % W
    rows = (slots[:, None] * s + torch.arange(s, device="cuda")).flatten()
    k8, ks = _quantise(_norm_rope(t["k"], t["kw"], rope, first, gh, gw).transpose(1, 2).contiguous(), s)
    v8, vs = _quantise(t["v"].float().transpose(1, 2).contiguous(), s)
    t["k8"].view(torch.uint8)[:, :, rows] = k8.view(torch.uint8)
    t["v8"].view(torch.uint8)[:, :, rows] = v8.view(torch.uint8)
    t["k_scale"][:, :, slots] = ks
    t["v_scale"][:, :, slots] = vs
    return t["k8"], t["v8"], t["k_scale"], t["v_scale"]


def _run_own(t):
    import static_sparse_attention_b200 as ra
    c = t["case"]
    if c["op"] == "attend":
        lse = torch.empty(c["B"], c["H"], c["nq"], device="cuda")
        o = ra.cache8_attention(t["q"], t["k8"], t["v8"], t["k_scale"], t["v_scale"], c["held"],
                                key_counts=t["counts"], lse=lse)
        return o, lse
    if c["op"] == "norm_rope":
        return ra.qk_norm_rope(t["q"], t["k"], t["qw"], t["kw"], rope=t["rope"], frame0=t["first"], eps=EPS)
    if c["op"] == "norm_rope_bwd":
        return ra.qk_norm_rope_bwd(t["q"], t["k"], t["dq"], t["dk"], t["qw"], t["kw"], rope=t["rope"],
                                   frame0=t["first"], eps=EPS)
    ra.cache8_append(t["k"], t["v"], t["k8"], t["v8"], t["k_scale"], t["v_scale"], c["frame"], t["kw"],
                     rope=t["rope"], eps=EPS)
    return t["k8"], t["v8"], t["k_scale"], t["v_scale"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    c = case
    if c["op"] == "attend":
        keys, row = sum(counts_of(c)) * c["H"], c["B"] * c["H"] * c["nq"]
        scales = sum(-(-n // c["s"]) * -(-c["s"] // BLOCK) for n in counts_of(c)) * c["H"]
        return dict(bytes=2 * keys * c["d"] + 8 * scales + row * (4 * c["d"] + 4), flops=4 * c["nq"] * keys * c["d"])
    tokens = c["B"] * (c["frames"] if c["op"] == "append" else c["f"]) * c["gh"] * c["gw"]
    if c["op"] == "append":
        e = tokens * c["H"] * c["d"]
        scales = c["B"] * c["frames"] * c["H"] * -(-(c["gh"] * c["gw"]) // BLOCK)
        return dict(bytes=6 * e + 8 * scales, flops=12 * e)
    e = tokens * (c["H"] + c["Hk"]) * c["d"]
    return dict(bytes=4 * e, flops=8 * e) if c["op"] == "norm_rope" else dict(bytes=6 * e, flops=18 * e)


# ------------------------------------------------- the definitions, in 64 bits
def _defined(x, w, rope, first, gh, gw):
    """[B, n, H, d] in 64 bits: the norm by the row's length, the rotation as a complex product."""
    B, n, H, d = x.shape
    if w is not None:
        x = x * w.double() / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + EPS)
    if rope is None:
        return x
    t, h, v = (torch.view_as_complex(r.double()) for r in rope)
    f = n // (gh * gw)
    turn = torch.cat([t[first:first + f, None, None, :].expand(f, gh, gw, -1), h[None, :, None, :].expand(f, gh, gw, -1),
                      v[None, None, :, :].expand(f, gh, gw, -1)], -1).reshape(1, n, 1, d // 2)
    return torch.view_as_real(torch.view_as_complex(x.reshape(B, n, H, d // 2, 2)) * turn).reshape(B, n, H, d)


def exact(case, seed):
    t = prepare(case, seed)
    c = t["case"]
    if c["op"] == "attend":
        o, lse = [], []
        for b, n in enumerate(counts_of(c)):
            for h in range(c["H"]):
                at = lambda code, scale: code[b, h, :n].double() * _per_token(scale[b, h].double(), c["s"])[:n]  # noqa: E731
                x = t["q"][b, h].double() @ at(t["k8"], t["k_scale"]).T / math.sqrt(c["d"])
                z = torch.logsumexp(x, -1)
                lse.append(z)
                o.append(torch.exp(x - z[:, None]) @ at(t["v8"], t["v_scale"]))
        shape = (c["B"], c["H"], c["nq"])
        return torch.stack(o).reshape(*shape, c["d"]), torch.stack(lse).reshape(shape)
    place = (t["rope"], t["first"], c["gh"], c["gw"])
    if c["op"] == "norm_rope":
        return [_defined(t[x].double(), t[x + "w"], *place).transpose(1, 2).contiguous() for x in ("q", "k")]
    if c["op"] == "norm_rope_bwd":
        out = {}
        for x in ("q", "k"):  # the chain rule of the definition itself
            at = t.pop(x).double().requires_grad_()
            w = t[x + "w"].double().requires_grad_() if t[x + "w"] is not None else None
            got = torch.autograd.grad(_defined(at, w, *place), [at] if w is None else [at, w],
                                      t.pop("d" + x).double().transpose(1, 2))
            out[x], out[x + "w"] = got[0], got[1] if w is not None else None
        return out["q"], out["k"], out["qw"], out["kw"]

    def held(x, s):
        """64-bit values [B, H, frames * s, d] -> the e4m3 values and scales that stand for them."""
        codes, scales = [], []
        for j in range(0, x.shape[2], s):
            row_codes, row_scales = [], []
            for i in range(j, j + s, BLOCK):
                part = x[:, :, i:min(i + BLOCK, j + s)]
                top = part.abs().amax((2, 3))
                k = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126)
                k = torch.where(top > 0, k, torch.zeros_like(k))
                k = torch.where(top > 448.0 * torch.exp2(k), k + 1, torch.where(top <= 224.0 * torch.exp2(k), k - 1, k))
                k = torch.where(top > 0, k.clamp(min=-126), torch.zeros_like(k))
                unit = torch.exp2(k)
                y = part / unit[:, :, None, None]
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                row_codes.append(torch.round(y / step) * step)
                row_scales.append(unit)
            codes.append(torch.cat(row_codes, 2))
            scales.append(torch.stack(row_scales, -1))
        return torch.cat(codes, 2), torch.stack(scales, 2)

    s = c["gh"] * c["gw"]
    k8, ks = held(_defined(t["k"].double(), t["kw"], *place).transpose(1, 2), s)
    v8, vs = held(t["v"].double().transpose(1, 2), s)
    rings = [t["k8"].float(), t["v8"].float(), t["k_scale"].double(), t["v_scale"].double()]
    for j in range(c["frames"]):
        slot = (c["frame"] + j) % c["W"]
        for ring, new in ((rings[0], k8), (rings[1], v8)):
            ring[:, :, slot * s:(slot + 1) * s] = new[:, :, j * s:(j + 1) * s]
        for ring, new in ((rings[2], ks), (rings[3], vs)):
            ring[:, :, slot] = new[:, :, j]
    return rings
