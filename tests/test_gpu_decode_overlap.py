"""GPU: outputs of the NVFP4 operators in the memory of their inputs.

The linear stores y while other CTAs read x: an overlap is refused.  The layer has read
all of x before it stores: in place it gives the same bits.
"""
import pytest
import torch

from tests.test_gpu_decode_fp4 import S, fp4, routes  # noqa: F401

pytestmark = pytest.mark.gpu


def test_linear_refuses_overlap(S):  # noqa: F811
    B = S.binding
    n, T = 256, 4
    gen = torch.Generator("cuda").manual_seed(1)
    c, s, g = fp4(gen, 1, n, n)
    lin = S.Fp4Linear(c[0], s[0], g)
    buf = torch.randn(4 * T * n, device="cuda", generator=gen).bfloat16()
    x = buf[T * n:2 * T * n].view(T, n)
    want = lin.forward(x.clone())

    def out(first):  # BF16 [T, n] from element `first` on
        return buf[first:first + T * n].view(T, n)

    before = buf.clone()
    wide = buf[:2 * T * n].view(T, 2 * n)[:, n:]             # rows apart, y over one of them
    for xs, o in ((x, x), (x, out(T * n - n)), (x, out(T * n + n)), (x, out(1)), (x, out(2 * T * n - 1)),
                  (wide, out(0)), (wide, out(2 * T * n - n)), (wide[:2], buf[3 * n - 2:5 * n - 2].view(2, n)),
                  (x, buf[:2 * T * n].view(torch.float32).view(T, n))):
        with pytest.raises(B.MoEError) as e:
            lin.forward(xs, out=o)
        assert e.value.status == B.MOE_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    for o in (out(0), out(2 * T * n)):                        # directly before and after x
        assert torch.equal(lin.forward(x, out=o), want)
    one = buf[:2 * n].view(2, n)
    lin.forward(one[:1], out=one[1:])                         # a single row beside its output
    assert torch.equal(one[1:], lin.forward(one[:1]))


@pytest.mark.parametrize("H,I,E,K", [(512, 256, 8, 2), (7168, 128, 40, 2), (16384, 256, 24, 2)])
def test_layer_in_place(S, H, I, E, K):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(H)
    layer = S.Fp4MoELayer(H, I, E, K)
    layer.bind_weights(*fp4(gen, E, 2 * I, H), *fp4(gen, E, H, I))
    for T in (1, 5, 16):
        x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
        idx, w = routes(gen, T, E, K)
        want = layer.forward(x, idx, w)
        for _ in range(5):
            y = x.clone()
            assert torch.equal(layer.forward(y, idx, w, out=y), want)
        idx[:] = -1
        assert not layer.forward(x, idx, w, out=x).any() and layer.read_status() == (0, 0)
