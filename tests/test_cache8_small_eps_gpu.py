"""Keys so small, normed with so small an eps, that the norm's factor and the scale's
would leave fp32 if they were multiplied first: what the append writes is still the
definition's."""
import pytest
import torch

from tests import _gpu, _heads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("eps", [1e-12, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("size", [1.0, 1e-10, 1e-20, 1e-30, 1e-37])
def test_append_of_small_keys(size, eps, d):
    _gpu.need_gpu()
    ra = _gpu.ra()
    B, H, s, W = 1, 2, 70, 2
    g = torch.Generator(device="cuda").manual_seed(d)
    k = (torch.randn(B, s, H, d, generator=g, device="cuda").sign() *
         (1 + torch.rand(B, s, H, d, generator=g, device="cuda")) * size).bfloat16()
    k[:, 5] = 0
    k[:, :, :, 7] = 0
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    cache = ra.SwcCache8(B, H, d, s, W)
    cache.append(k, k, w, eps=eps)
    assert ra.device_status() == ra.RA_OK
    eps = torch.tensor(eps, dtype=torch.float32).double().item()  # as the call rounds it
    k64, bound = _heads.norm_rope(k, w, None, 0, eps)
    # fp32 on the way, not bf16: the row's error; and where x^2 leaves fp32's normal range,
    # the mean's: half the least step, 2^-150, in each of the mean, the product with 1 / d and
    # the sum with eps, or all of a mean that vanishes; half of that relative error is r's
    mean = k.double().cpu().square().mean(-1, keepdim=True).transpose(1, 2)
    lost = torch.minimum(torch.full_like(mean, 3 * 2.0 ** -150), 2 * mean) / (mean + eps) / 2
    bound = k64.abs() * (_heads.ROW + lost)
    scale = cache.k_scale[:, :, :1].double().cpu()
    low, high = _heads.block_scales(k64.abs() - bound, s), _heads.block_scales(k64.abs() + bound, s)
    assert bool(((scale >= low) & (scale <= high)).all())
    unit = _heads.per_token(scale, s)
    got = cache.k8[:, :, :s].float().double().cpu()
    assert not bool(torch.isnan(got).any())
    low, high = _heads.e4m3((k64 - bound) / unit), _heads.e4m3((k64 + bound) / unit)
    assert bool(((got >= low) & (got <= high)).all())
    assert bool((got[:, :, 5] == 0).all()) and bool((got[..., 7] == 0).all())
