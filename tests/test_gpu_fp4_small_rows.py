"""GPU: rows of x (or of h) so small, or matrix scales so far from one, that the product of a
row's scale and the matrix's is no normal number, although the result is one.
"""
import math

import pytest
import torch

from tests.test_gpu_decode_fp4 import S, fp4, layer64, value64  # noqa: F401

pytestmark = pytest.mark.gpu


def ones_to_twos(gen, *shape):
    """Magnitudes in [1, 2) and signs: BF16 values that any normal power of two scales exactly."""
    x = 1 + torch.randint(0, 128, shape, device="cuda", generator=gen).float() / 128
    return torch.where(torch.rand(*shape, device="cuda", generator=gen) < 0.5, x, -x)


@pytest.mark.parametrize("rows,cols", [(64, 64), (130, 1408), (4096, 512)])
@pytest.mark.parametrize("T", [3, 16])
def test_linear_scales_exactly(S, rows, cols, T):  # noqa: F811
    """y of x * 2^k is y of x times 2^k, bit for bit, while both are normal."""
    gen = torch.Generator("cuda").manual_seed(rows)
    c, s, g = fp4(gen, 1, rows, cols)
    lin = S.Fp4Linear(c[0], s[0], g)
    x = ones_to_twos(gen, T, cols)
    y = lin.forward(x.bfloat16(), out_dtype=torch.float32).double()
    for k in (-40, -100, -112, -115, -118, 100, 110):
        z = lin.forward((x * 2.0**k).bfloat16(), out_dtype=torch.float32).double()
        want = y * 2.0**k
        assert torch.all((z == want) | (want.abs() < 2.0**-126))
        assert torch.all((z - want).abs() <= 2.0**-149)


@pytest.mark.parametrize("k,gk", [(-110, 100), (-60, 60), (-115, 30), (100, -100), (60, -110), (-100, 0), (0, -110)])
def test_linear_with_far_matrix_scales(S, k, gk):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(k + 200)
    c, s, g = fp4(gen, 1, 96, 256)
    g = g * 2.0**gk
    lin = S.Fp4Linear(c[0], s[0], g)
    x = (ones_to_twos(gen, 5, 256) * 2.0**k).bfloat16()
    w = value64(c[0], s[0], g)
    ref, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    y = lin.forward(x, out_dtype=torch.float32)
    # a float sum of 256 products, and one subnormal step
    assert torch.all((y.double() - ref).abs() <= (256 / 16 + 32) * 2.0**-23 * mag + 2.0**-149)


@pytest.mark.parametrize("T", [1, 5, 16])
def test_layer_with_small_h(S, T):  # noqa: F811
    """x near 2^-57 leaves h near 2^-113, and W2's scale is 2^-25: outputs near 2^-122, normal
    in BF16.  The bound is the layer's (8 bits of the output, 11 of h), without an absolute term
    but BF16's smallest step, 2^-133."""
    H, I, E, K = 512, 256, 8, 2
    gen = torch.Generator("cuda").manual_seed(T)
    p1 = fp4(gen, E, 2 * I, H)
    c, s, _ = fp4(gen, E, H, I, lo=0x70, hi=0x7F)
    p2 = c, s, (1.05 + 0.9 * torch.rand(E, device="cuda", generator=gen)) * 2.0**-25
    layer = S.Fp4MoELayer(H, I, E, K)
    layer.bind_weights(*p1, *p2)
    idx = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:K] for _ in range(T)]).int()
    w = 1 + torch.rand(T, K, device="cuda", generator=gen)
    x = (ones_to_twos(gen, T, H) * 2.0**-57).bfloat16()
    y = layer.forward(x, idx, w)
    assert layer.read_status() == (0, 0)
    ref, mag = layer64(p1, p2, x, idx, w, E, I)
    assert ref.abs().median() > 2.0**-126
    bound = 2.0**-8 * (1 + 2.0**-8) * ref.abs() + 2.0**-11 * mag + 2.0**-133
    assert torch.all((y.double() - ref).abs() <= bound)
