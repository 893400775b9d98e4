"""GPU: moe_fp4_forward where the token rows do not all fit in shared memory.

There the kernel divides its shared memory by the routes: few tokens per expert
leave more room to the weights' copies, more of them to the rows.  Both
divisions, their border and experts that take several sweeps, against float64.
"""
import pytest
import torch

from tests.test_gpu_decode_fp4 import S, check_layer, fp4, routes  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,I,E,K", [(7168, 128, 64, 2), (16384, 256, 24, 2), (5120, 1536, 40, 4), (4096, 128, 128, 8)])
@pytest.mark.parametrize("T", [7, 11, 16])
def test_random(S, H, I, E, K, T):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(H + T)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    check_layer(S, p1, p2, x, *routes(gen, T, E, K))


@pytest.mark.parametrize("shared", range(0, 17, 2))
def test_crowds(S, shared):  # noqa: F811
    """`shared` tokens on one pair of experts, the others apart: one handle over all."""
    H, I, E, K, T = 7168, 128, 40, 2, 16
    gen = torch.Generator("cuda").manual_seed(7)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    w = torch.rand(T, K, device="cuda", generator=gen)
    idx = torch.arange(T * K, dtype=torch.int32, device="cuda").view(T, K) + 2
    idx[:shared, 0], idx[:shared, 1] = 37, 1
    y, layer = check_layer(S, p1, p2, x, idx, w)
    spread = torch.arange(T * K, dtype=torch.int32, device="cuda").view(T, K)
    check_layer(S, p1, p2, x, spread, w, layer=layer)
    assert torch.equal(layer.forward(x, idx, w), y)
