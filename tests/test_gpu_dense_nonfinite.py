"""Infinities and NaN in the inputs of the dense products: they show in their own rows of the
output, as NaN, and nowhere else."""
import math

import pytest
import torch

from tests.test_gpu_dense import BF, HF, S, mlp_case, rand, weights8  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 16, 60, 130, 600])
@pytest.mark.parametrize("bad", [[math.inf], [-math.inf], [math.inf, math.nan], [math.nan, -math.inf, math.inf]])
def test_linear_rows_with_infinities(S, T, bad):
    """Up to 16 rows are rounded where they are multiplied, more by a kernel of their own."""
    codes, scales = weights8(384, 384, seed=5)
    lin = S.Fp8Linear(codes, scales, max_tokens=T + 2)
    x = rand(T, 384, seed=6)
    want = lin.forward(x)
    t = T // 2
    x[t, 200:200 + len(bad)] = torch.tensor(bad, dtype=BF, device="cuda")
    for dtype in (BF, torch.float32):
        got = lin.forward(x, out_dtype=dtype)
        rows = torch.arange(T, device="cuda") != t
        assert torch.equal(got[rows].to(BF), want[rows]) and got[t].isnan().all()


def test_linear_largest_finite_values_stay_numbers(S):
    """Next to infinity: BF16's largest number is rounded to 256 * 2^120."""
    codes, scales = weights8(256, 256, seed=7)
    codes.fill_(0)
    codes[:, 3] = 0x30  # 0.5
    scales.fill_(2.0 ** -8)
    for T in (4, 40):
        x = torch.zeros(T, 256, dtype=BF, device="cuda")
        x[:, 3] = 3.3895313892515355e38
        got = S.Fp8Linear(codes, scales, max_tokens=T).forward(x, out_dtype=torch.float32)
        assert (got == 2.0 ** (128 - 1 - 8)).all()


@pytest.mark.parametrize("T", [3, 20, 100, 400])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype,act", [(BF, "silu"), (HF, "gelu")])
def test_mlp_rows_with_infinities(S, T, bad, dtype, act):
    """Gates of both infinities: act(-inf) is -inf * 0, so the row's sums are NaN."""
    w1, w2, x, mlp = mlp_case(S, T, 264, 136, dtype, act)
    saved, dy = torch.empty(T, 272, device="cuda"), rand(T, 264, seed=8, dtype=dtype)
    want = mlp.forward(x, saved=saved)
    want_dx = mlp.backward(dy, x, saved)[0]
    t = T - 2
    x[t, 3] = bad
    saved2 = torch.empty_like(saved)
    got = mlp.forward(x, saved=saved2)
    rows = torch.arange(T, device="cuda") != t
    assert torch.equal(got[rows], want[rows]) and got[t].isnan().all()
    assert torch.equal(saved2[rows], saved[rows]) and not saved2[t].isfinite().any()
    dx, dw1, dw2 = mlp.backward(dy, x, saved2)
    assert torch.equal(dx[rows], want_dx[rows]) and dx[t].isnan().all()
    assert dw2.isnan().any() and dw1.isnan().any()  # sums over the rows: the bad one is among them
    dy[t, 5] = bad
    dx = mlp.backward(dy, x, saved)[0]  # (finite gate and up)
    assert torch.equal(dx[rows], want_dx[rows]) and not dx[t].isfinite().any()
