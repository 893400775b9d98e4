"""Waits of the CTA pairs that run out: a copy of the first pair never comes, the launch ends within
its limit, says so, leaves that pair's tiles unwritten, and the GPU and the object stay usable."""
import pytest
import torch

from tests import dense_choices as c
from tests import dense_reference as ref
from tests.test_gpu_dense import BF, F32, HF, S, mlp_case, rand, weights8  # noqa: F401

pytestmark = pytest.mark.gpu


def late(B, obj):
    """It timed out since the last read, and not since this one."""
    assert obj.read_status() == (B.MOE_ERR_DEVICE_TIMEOUT, B.MOE_DEV_TIMEOUT)
    assert obj.read_status() == (B.MOE_OK, 0)


@pytest.mark.parametrize("T,rows,cols", [(2710, 780, 128), (808, 3760, 128), (1031, 3873, 256), (2500, 3000, 640),
                                         (3084, 3277, 1664)])
def test_linear_on_pairs(S, T, rows, cols):
    B = S.binding
    codes, scales = weights8(rows, cols, seed=1)
    x = rand(T, cols, seed=2)
    xq, xs = ref.quantize_rows(x)
    slow, lin = (S.Fp8Linear(codes, scales, max_tokens=T, watchdog_test=w) for w in (True, False))
    assert slow.plan(T)["pairs"] and slow.plan(T, quantized=True)["pairs"]
    want = lin.forward(x, out_dtype=F32)
    ref.check(want, ref.linear(xq, xs, codes, scales, F32))
    for call in (lambda o: slow.forward(x, out=o), lambda o: slow.forward_quantized(xq, xs, out=o)):
        out = torch.full_like(want, 7.0)
        call(out)
        late(B, slow)
        assert out[0, 0] == 7 and not (out == 7).all()
    assert torch.equal(lin.forward(x, out_dtype=F32), want) and lin.read_status() == (B.MOE_OK, 0)


@pytest.mark.parametrize("T,H,I,dtype,act", [(3343, 1024, 864, BF, "silu"), (4100, 1032, 1000, HF, "gelu"),
                                             (1954, 520, 1544, BF, "gelu")])
def test_block_on_pairs(S, T, H, I, dtype, act):
    """Each of the block's launches: gate by what it leaves unwritten, dh as the only launch of a
    call, and the last ones as the only ones that withhold a copy."""
    B = S.binding
    w1, w2, x, mlp = mlp_case(S, T, H, I, dtype, act, seed=3)
    plan = mlp.plan(T)
    on_pairs = {n for n in c.LAUNCHES if plan[n]["pairs"]}
    assert on_pairs >= {"gate", "dh", "gradients"}
    dy = rand(T, H, seed=4, dtype=dtype, scale=0.25)
    want_saved = torch.empty(T, 2 * I, device="cuda")
    want = mlp.forward(x, saved=want_saved)
    want_grads = mlp.backward(dy, x, want_saved)

    slow = S.GatedMlp(w1, w2, max_tokens=T, activation=act, watchdog_test=True)
    saved = torch.full_like(want_saved, 7.0)
    slow.forward(x, saved=saved)
    late(B, slow)
    assert saved[0, 0] == 7 and (saved == want_saved).any()
    slow.backward(dy, x, want_saved, out=(None, None, None))
    late(B, slow)

    last = S.GatedMlp(w1, w2, max_tokens=T, activation=act, watchdog_last_test=True)
    saved.fill_(7.0)
    y = torch.full_like(want, 7.0)
    last.forward(x, out=y, saved=saved)
    late(B, last)
    assert torch.equal(saved, want_saved)
    if "down" in on_pairs:
        assert y[0, 0] == 7 and (y == want).any()
    last.backward(dy, x, saved, out=(None, None, None))
    assert last.read_status() == (B.MOE_OK, 0)
    grads = [torch.full_like(t, 7.0) for t in want_grads]
    last.backward(dy, x, saved, out=grads)
    late(B, last)
    assert sum(int((a == 7).sum() >= 64 * 256) for a in grads) >= 1  # the first pair's tiles

    assert torch.equal(mlp.forward(x), want) and mlp.read_status() == (B.MOE_OK, 0)
    assert all(torch.equal(a, b) for a, b in zip(mlp.backward(dy, x, want_saved), want_grads))
