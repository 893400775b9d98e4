"""GPU: moe_add_rms_norm takes every static scale that is positive and finite, as the
layer's set_activation_scales does: code = E4M3_RNE_sat(y * float(1 / scale))."""
import pytest
import torch

from tests.test_gpu_decode_fp4 import S  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0**-126, 2.0**-100, 2.9e38, 3.2e38, torch.finfo(torch.float32).max])
def test_codes(S, scale):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(1)
    H = 256
    # y near the scale's size: one row, normed to about 1, times a weight of that size
    x = torch.randn(3, H, device="cuda", generator=gen).bfloat16()
    w = torch.full((H,), min(scale, 1e38), device="cuda").bfloat16()
    y, _, q, s = S.add_rms_norm(x, w, fmt="per_tensor", scale=scale)
    x64 = x.double()
    y64 = x64 / (x64.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    t = y64 / scale
    v = q.view(torch.float8_e4m3fn).double()
    # E4M3: four significant bits, half of 2^-9 below; 1 / scale may be subnormal (2^-23 of it and more
    # for the largest scales: 2^-21)
    assert s is None and torch.all((v - t).abs() <= (2.0**-4 + 2.0**-10) * t.abs() + 2.0**-10)
    assert v.abs().max() > 0.125
