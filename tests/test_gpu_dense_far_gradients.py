"""Derivatives of the activations at the ends of FP32's range: 0 on the left, 1 on the right."""
import pytest
import torch

from tests.test_gpu_dense import BF, S  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,I", [(3, 136), (140, 136), (3393, 688)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_up_to_the_largest_number(S, T, I, act):
    """dx is dg itself (the gate's rows are the identity, up's are zero): dh * u * act'(g) with powers of two
    for dh and u, so exact."""
    H = I
    w1 = torch.zeros(2 * I, H, dtype=BF, device="cuda")
    w1[:I].fill_diagonal_(1.0)
    w2 = torch.eye(H, I, dtype=BF, device="cuda")
    size = torch.tensor([1e4, 1e12, 1e19, 1e30, 1e36, 3e36, 4e36, 1e37, 1e38, 3e38, 3.4e38], device="cuda")
    g = torch.cat((-size, size)).repeat(T * I // 22 + 1)[:T * I].view(T, I)
    u = torch.exp2(torch.arange(T * I, device="cuda") % 5 - 2.0).view(T, I)
    dy = torch.exp2(-(torch.arange(T * H, device="cuda") % 7) - 10.0).view(T, H).to(BF)
    mlp = S.GatedMlp(w1, w2, max_tokens=T, activation=act)
    dx = torch.empty(T, H, dtype=BF, device="cuda")
    mlp.backward(dy, torch.zeros_like(dx), torch.cat((g, u), -1), out=(dx, None, None))
    want = torch.where(g > 0, dy.float() * u, 0.0)
    assert torch.equal(dx.float(), want)
