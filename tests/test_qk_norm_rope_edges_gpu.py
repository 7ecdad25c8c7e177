"""Norm and rotation of Q and K where values are not finite: what is not rotated is not
touched by the channel beside it."""
import math

import pytest
import torch

from tests import _gpu, _heads

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def _same(got, want):
    """Equal, NaN where NaN is wanted."""
    got, want = got.double().cpu(), want.double().cpu()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("d", [64, 128])
def test_channels_that_are_not_rotated_keep_their_values(d):
    """Axes of 2, 4 and 4 channels: the others of a rotated row go through as they are,
    infinities and NaN too, forward and backward."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    gh, gw, H = 3, 4, 5
    n = 2 * gh * gw
    rope = ra.rope3d(2, gh, gw, d, axes=(2, 4, 4))
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(1, n, H, d, generator=g, device="cuda").bfloat16()
    for i, (at, value) in enumerate(((10, INF), (11, -INF), (12, NAN), (d - 1, INF), (d - 2, NAN), (17, -INF))):
        x[0, i::7, :, at] = value
    y, _ = ra.qk_norm_rope(x, rope=rope)
    assert _same(y[..., 10:], x.transpose(1, 2)[..., 10:])
    assert bool(torch.isfinite(y[..., :10]).all())
    dy = x.transpose(1, 2).contiguous()
    dx, _, _, _ = ra.qk_norm_rope_bwd(torch.zeros_like(x), None, dy, None, rope=rope)
    assert _same(dx[..., 10:], x[..., 10:])
    assert bool(torch.isfinite(dx[..., :10]).all())


@pytest.mark.parametrize("rotated", [False, True])
def test_an_infinity_in_a_normed_row(rotated):
    """The row's norm is infinite: finite values over it are 0 and the infinity itself
    has no value; the channel beside it has its 0 where nothing is rotated."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    d, w = 64, torch.ones(64, device="cuda")
    x = torch.ones(1, 4, 2, d, device="cuda").bfloat16()
    x[0, 2, 1, 33] = INF
    rope = ra.rope3d(1, 2, 2, d, axes=(2, 4, 4)) if rotated else None
    y, _ = ra.qk_norm_rope(x, None, w, rope=rope)
    want = torch.zeros(d)
    want[33] = NAN
    assert _same(y[0, 1, 2], want)
    assert bool(torch.isfinite(y[0, 0]).all()) and bool(torch.isfinite(y[0, 1, [0, 1, 3]]).all())


@pytest.mark.parametrize("eps", [1e-12, 1e-38, 1e-44])
def test_gradient_of_zero_and_small_rows_with_a_small_eps(eps):
    """The norm's factor is up to 2^75, its square no fp32 number: rows of zeros have the
    gradient dy * w / sqrt(eps), small rows the formula's."""
    _gpu.need_gpu()
    ra = _gpu.ra()
    d = 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, 6, 2, d, generator=g, device="cuda").bfloat16()
    x[0, 1] = 0
    x[0, 2] *= 1e-15
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    dy = (torch.randn(1, 2, 6, d, generator=g, device="cuda") * 1e-6).bfloat16()
    dx, _, dw, _ = ra.qk_norm_rope_bwd(x, None, dy, None, w, eps=eps)
    eps = torch.tensor(eps, dtype=torch.float32).double().item()  # as the call rounds it
    want, bound, dw64, dw_bound = _heads.norm_rope_bwd(x, dy, w, None, 0, eps)
    assert bool(((dx.double().cpu() - want).abs() <= bound).all())
    assert bool(((dw.double().cpu() - dw64).abs() <= dw_bound).all())
