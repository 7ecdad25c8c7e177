"""Plain 64-bit forms of the per-head norm, the 3-axis rotation, their gradient
and the e4m3 block quantiser, written from the formulas with torch on the CPU,
and the rounding bounds that the GPU tests hold the kernels to."""
import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2   # a rounding to bf16 is off by at most this, relative
U32 = torch.finfo(torch.float32).eps / 2     # and one to fp32 by this
# A row's sums (mean of squares, mean of products) add at most 128 terms in fp32,
# each addition off by U32 of the partial sum: 128 * U32 relative to the sum of
# magnitudes; the few roundings beside them are counted in with 32 more.
ROW = 160 * U32


def table64(length, pairs, base=10000.0, start=0):
    """(cos, sin) in fp64, [length, pairs, 2]"""
    p = torch.arange(start, start + length, dtype=torch.float64)[:, None]
    i = torch.arange(pairs, dtype=torch.float64)[None, :]
    a = p * base ** (-i / max(pairs, 1))
    return torch.stack([a.cos(), a.sin()], -1)


def angles(rope, frame0, n, d):
    """cos, sin [n, d / 2] in fp64 from the three tables (unrotated pairs: 1, 0)."""
    t, h, w = (x.double().cpu() for x in rope)
    i = torch.arange(n)
    s = h.shape[0] * w.shape[0]
    at = torch.cat([t[frame0 + i // s], h[i % s // w.shape[0]], w[i % s % w.shape[0]]], 1)
    rest = torch.tensor([1.0, 0.0], dtype=torch.float64).expand(n, d // 2 - at.shape[1], 2)
    at = torch.cat([at, rest], 1)
    return at[..., 0], at[..., 1]


def rotate(x, cos, sin):
    """x [B, n, H, d], cos and sin [n, d / 2]"""
    a, b = x[..., 0::2], x[..., 1::2]
    cos, sin = cos[None, :, None, :], sin[None, :, None, :]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def norm_rope(x, weight, rope, frame0, eps):
    """x [B, n, H, d] of any type -> ([B, H, n, d] in fp64, bound of an fp32 computation rounded to bf16)"""
    x = x.double().cpu()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double().cpu()
    # each output is a sum of two products of fp32 values that carry the row's error
    size = (x[..., 0::2].abs() + x[..., 1::2].abs()).repeat_interleave(2, -1)
    y = x
    if rope is not None:
        y = rotate(x, *angles(rope, frame0, x.shape[1], x.shape[3]))
    bound = y.abs() * BF16 + size * ROW + 1e-38
    return y.transpose(1, 2), bound.transpose(1, 2)


def norm_rope_bwd(x, dy, weight, rope, frame0, eps):
    """(dx [B, n, H, d], its bound, dweight, its bound) in fp64"""
    x, g = x.double().cpu(), dy.double().cpu().transpose(1, 2)
    size = (g[..., 0::2].abs() + g[..., 1::2].abs()).repeat_interleave(2, -1)  # of g before the rotation's cancellation
    if rope is not None:
        cos, sin = angles(rope, frame0, x.shape[1], x.shape[3])
        g = rotate(g, cos, -sin)
    if weight is None:
        return g, g.abs() * BF16 + size * ROW + 1e-38, None, None
    w = weight.double().cpu()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    xh, a = x * r, g * w
    c = (a * xh).mean(-1, keepdim=True)
    dx = r * (a - xh * c)
    whole = r * (size * w.abs() + xh.abs() * (size * w.abs() * xh.abs()).mean(-1, keepdim=True))
    dw = (g * xh).sum((0, 1, 2))
    rows = x[..., 0].numel()  # every addition of dw, and the row's own error, relative to the sum of magnitudes
    dw_bound = (size * xh.abs()).sum((0, 1, 2)) * (ROW + rows * U32)
    return dx, dx.abs() * BF16 + whole * 2 * ROW + 1e-38, dw, dw_bound


def block_scales(x, s, block=64):
    """x fp64 [B, H, frames * s, d] -> scales [B, H, frames, blocks]: the least power of
    two (not below 2^-126) that brings the block's largest value to at most 448; 1 for zeros."""
    B, H, n, d = x.shape
    out = []
    for f in range(n // s):
        row = []
        for i in range(f * s, (f + 1) * s, block):
            top = x[:, :, i:min(i + block, (f + 1) * s)].abs().amax((2, 3))
            m, e = torch.frexp(top)
            k = (e - 9 + (m > 0.875)).clamp(min=-126).double()
            row.append(torch.where(top > 0, torch.exp2(k), torch.ones_like(top)))
        out.append(torch.stack(row, -1))
    return torch.stack(out, 2)


def per_token(scale, s, block=64):
    """[B, H, frames, blocks] -> [B, H, frames * s, 1]"""
    B, H, f, _ = scale.shape
    return scale.repeat_interleave(block, -1)[..., :s].reshape(B, H, f * s, 1)


def e4m3(x):
    """Nearest e4m3 value (ties to even) of fp64 x, |x| <= 448 after rounding."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step
