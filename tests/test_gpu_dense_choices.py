"""Every kernel, tile width and share of K of the dense products on the GPU: the sizes of
dense_choices.py are divided as it says, and the results are right element by element and in norm."""
import pytest
import torch

from tests import dense_choices as c
from tests import dense_norms as norms
from tests import dense_reference as ref
from tests.test_gpu_dense import BF, F32, HF, S, mlp_case, rand, weights8  # noqa: F401

pytestmark = pytest.mark.gpu

SMS = 152


def choice_holds():
    return torch.cuda.get_device_properties(0).multi_processor_count == SMS


@pytest.mark.parametrize("row", c.MLP, ids=lambda r: "-".join(map(str, r[:3])))
def test_mlp_plans(S, row):
    T, H, I, *want = row
    _, _, _, mlp = mlp_case(S, T, H, I, BF, "silu")
    plan = mlp.plan(T)
    if choice_holds():
        assert [c.launch(plan[n]) for n in c.LAUNCHES] == want
    assert plan == S.GatedMlp(*mlp.weights, max_tokens=T + 1).plan(T)
    assert all(v == 0 for p in mlp.plan(0).values() for v in p.values())
    for bad, status in ((-1, S.binding.MOE_ERR_INVALID_ARG), (T + 1, S.binding.MOE_ERR_CAPACITY)):
        with pytest.raises(S.binding.MoEError) as e:
            mlp.plan(bad)
        assert e.value.status == status


@pytest.mark.parametrize("row", c.LINEAR, ids=lambda r: "-".join(map(str, r[:3])))
def test_linear_plans(S, row):
    T, rows, cols, want = row
    lin = S.Fp8Linear(*weights8(rows, cols), max_tokens=T)
    if choice_holds():
        assert c.launch(lin.plan(T)) == c.launch(lin.plan(T, quantized=True)) == want
    assert not any(lin.plan(0).values())
    for bad, status in ((-1, S.binding.MOE_ERR_INVALID_ARG), (T + 1, S.binding.MOE_ERR_CAPACITY)):
        with pytest.raises(S.binding.MoEError) as e:
            lin.plan(bad)
        assert e.value.status == status


@pytest.mark.parametrize("row", c.MLP, ids=lambda r: "-".join(map(str, r[:3])))
@pytest.mark.parametrize("dtype,act,saved_type", [(BF, "silu", F32), (HF, "gelu", HF)])
def test_mlp_choices(S, row, dtype, act, saved_type):
    T, H, I = row[:3]
    w1, w2, x, mlp = mlp_case(S, T, H, I, dtype, act, seed=100)
    saved = torch.full((T + 2, 2 * I), 7.0, dtype=saved_type, device="cuda")
    y = mlp.forward(x, saved=saved[1:-1])
    assert (saved[0] == 7).all() and (saved[-1] == 7).all()
    saved = saved[1:-1]
    want = ref.forward(x, w1, w2, act, dtype)
    ref.check(y, want, "y")
    norms.check(y, want[0], norms.rounded(dtype), "y")
    gu = x.double() @ w1.double().t()
    norms.check(saved, gu, norms.rounded(saved_type) + norms.summed(H, 16), "saved")
    dy = rand(T, H, seed=105, dtype=dtype, scale=0.25)
    for grad_type in (dtype, F32):
        out = [torch.full((n + 2, m), 7.0, dtype=t, device="cuda") for n, m, t in
               ((T, H, dtype), (2 * I, H, grad_type), (H, I, grad_type))]
        grads = mlp.backward(dy, x, saved, out=[t[1:-1] for t in out])
        for n, got, w in zip(("dx", "dw1", "dw2"), grads, ref.backward(dy, x, saved, w1, w2, act, dtype, grad_type)):
            ref.check(got, w, n)
            norms.check(got, w[0], norms.rounded(dtype), n)
        assert all((t[0] == 7).all() and (t[-1] == 7).all() for t in out)
    assert mlp.read_status() == (0, 0)


@pytest.mark.parametrize("row", c.LINEAR, ids=lambda r: "-".join(map(str, r[:3])))
def test_linear_choices(S, row):
    """Weights of one scale, so that every block of K counts alike."""
    T, rows, cols = row[:3]
    codes, scales = weights8(rows, cols, seed=110)
    scales.fill_(2.0 ** -8)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    x = rand(T, cols, seed=111)
    xq, xs = ref.quantize_rows(x)
    for dtype in (F32, BF):
        want = ref.linear(xq, xs, codes, scales, dtype)
        for got in (lin.forward(x, out_dtype=dtype), lin.forward_quantized(xq, xs, out_dtype=dtype)):
            ref.check(got, want)
            norms.check(got, want[0], norms.summed(cols) + (norms.rounded(BF) if dtype is BF else 0.0))
    assert lin.read_status() == (0, 0)


def test_linear_plan_at_the_limits(S):
    """2^24 tokens and rows: more tiles than 32 bits hold."""
    n = 1 << 24
    codes, scales = torch.zeros(n, 128, dtype=torch.uint8, device="cuda"), torch.ones(n // 128, 1, device="cuda")
    lin = S.Fp8Linear(codes, scales, max_tokens=n)
    for quantized in (False, True):
        p = lin.plan(n, quantized)
        area = 256 * p["width"] if p["pairs"] else 128 * p["width"]
        assert p["tiles"] * area >= n * n and p["tiles"] >= 2 ** 32
