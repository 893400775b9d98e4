"""The dense products on whole numbers, where every sum is exact in FP32 however it is
divided or truncated: results are equal, so a lost, doubled or misplaced term of any K shows."""
import pytest
import torch

from tests import dense_choices as c
from tests import dense_reference as ref
from tests.test_gpu_dense import BF, F32, HF, S  # noqa: F401

pytestmark = pytest.mark.gpu


def generator(*key):
    return torch.Generator("cuda").manual_seed(sum(k * 7919 ** i for i, k in enumerate(key)) % 2 ** 31)


def integers(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, device="cuda", generator=g).float()


LINEAR = [r[:3] for r in c.LINEAR] + [(1, 300, 32768), (15, 520, 16384), (33, 130, 32768), (129, 257, 7168), (700, 640, 7168),
                                      (2100, 1100, 1664), (8, 4096, 7168), (512, 512, 4992)]


@pytest.mark.parametrize("T,rows,cols", LINEAR)
def test_linear(S, T, rows, cols):
    """Values from -3 to 3 (weights by scales of 1 and 1/2): sums below 2^19
    in halves."""
    g = generator(T, rows, cols)
    w = integers(g, -3, 3, rows, cols)
    codes = w.to(torch.float8_e4m3fn).view(torch.uint8)
    scales = 0.5 + 0.5 * integers(g, 0, 1, (rows + 127) // 128, cols // 128)
    x = integers(g, -3, 3, T, cols).to(BF)
    s = scales.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)
    want = x.double() @ (w.double() * s).t()
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    xq, xs = ref.quantize_rows(x)
    for dtype in (F32, BF):
        exact = want.float().to(dtype)
        assert torch.equal(lin.forward(x, out_dtype=dtype), exact)
        assert torch.equal(lin.forward_quantized(xq, xs, out_dtype=dtype), exact)


MLP = [r[:3] for r in c.MLP] + [(1, 16384, 4096), (13, 2048, 20000), (100, 7168, 512), (700, 4096, 72), (129, 1000, 600)]


@pytest.mark.parametrize("T,H,I", MLP)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gate_and_up(S, T, H, I, dtype):
    """What the forward saves: sums of values from -3 to 3."""
    g = generator(T, H, I, 1)
    w1, x = integers(g, -3, 3, 2 * I, H).to(dtype), integers(g, -3, 3, T, H).to(dtype)
    saved = torch.empty(T, 2 * I, device="cuda")
    S.GatedMlp(w1, torch.zeros(H, I, dtype=dtype, device="cuda"), max_tokens=T).forward(x, saved=saved)
    assert torch.equal(saved, (x.double() @ w1.double().t()).float())


@pytest.mark.parametrize("T,H,I", MLP)
@pytest.mark.parametrize("dtype,act,saved_type", [(BF, "silu", F32), (HF, "gelu", HF), (BF, "gelu", BF)])
def test_block_and_gradients(S, T, H, I, dtype, act, saved_type):
    """Gates of 128, where the activation is the identity and its derivative 1 (what it is short
    of, far below half a step, goes in the rounding), one +-1 in each row of up, the
    rest from -1 to 1: h is +-128 or 0, and dg, du are whole numbers of 8 bits (times 128)."""
    g = generator(T, H, I, 2)
    x = integers(g, -1, 1, T, H)
    x[:, 0] = 1
    w1 = torch.zeros(2 * I, H, device="cuda")
    w1[:I, 0] = 128
    w1[I:].scatter_(1, torch.randint(0, H, (I, 1), device="cuda", generator=g), 2 * integers(g, 0, 1, I, 1) - 1)
    w2, dy = integers(g, -1, 1, H, I), integers(g, -1, 1, T, H)
    dy *= torch.rand(T, H, device="cuda", generator=g) < 1600 / H  # (dh below 2^8)
    x, w1, w2, dy = (t.to(dtype) for t in (x, w1, w2, dy))
    xd, w1d, w2d, dyd = (t.double() for t in (x, w1, w2, dy))
    gate, up = (xd @ w1d.t()).chunk(2, -1)
    h, dh = gate * up, dyd @ w2d
    assert (gate == 128).all() and up.abs().max() <= 1 and dh.abs().max() <= 256
    dgu = torch.cat((dh * up, dh * gate), -1)
    want = h @ w2d.t(), dgu @ w1d, dgu.t() @ xd, dyd.t() @ h
    assert all(w.abs().max() < 2.0 ** 30 for w in want) and want[2][:I].abs().max() < 2 ** 23
    mlp = S.GatedMlp(w1, w2, max_tokens=T, activation=act)
    saved = torch.empty(T, 2 * I, dtype=saved_type, device="cuda")
    y = mlp.forward(x, saved=saved)
    assert torch.equal(saved.double(), torch.cat((gate, up), -1))
    assert torch.equal(y, want[0].float().to(dtype))
    grads = mlp.backward(dy, x, saved)
    assert all(torch.equal(a, w.float().to(dtype)) for a, w in zip(grads, want[1:]))
    out = [None, *(integers(g, -3, 3, *w.shape) * 128 for w in want[2:])]
    old = [t.double() for t in out[1:]]
    mlp.backward(dy, x, saved, out=out, accumulate=True)
    assert all(torch.equal(a, (w + o).float()) for a, w, o in zip(out[1:], want[2:], old))
