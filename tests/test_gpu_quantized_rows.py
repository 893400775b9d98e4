"""GPU: moe_forward_quantized, and the norm's 8-bit output as its input.

The layer's own quantisation of a BF16 x and the codes and scales of the same
values given from outside must lead to the same bits.  The values of y are
BF16 here where the two are compared (the norm rounds the float y once, the
layer a BF16 y: their codes may differ by one step, so the norm's codes are
compared through the layer fed with the very values that they stand for,
which BF16 holds exactly: 4 significant bits times a power of two).
"""
import numpy as np
import pytest
import torch

from tests import gpu_harness as gh
from tests.test_gpu_parity import small_problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    import __graft_entry__ as ge
    ge.build()
    import serving_route_gb300
    return serving_route_gb300


def layer(S, H, I, E, K, T, fmt, w1, w2, **kw):
    q1, s1 = S.MegaMoELayer.quantize_weights(torch.from_numpy(w1).cuda(), fmt=fmt)
    q2, s2 = S.MegaMoELayer.quantize_weights(torch.from_numpy(w2).cuda(), fmt=fmt)
    m = S.MegaMoELayer(H, I, E, K, max_rows=T, fmt=fmt, **kw)
    m.bind_weights(q1, s1, q2, s2)
    if fmt == "per_tensor":
        m.set_activation_scales(*SCALES)
    return m


SCALES = (0.015625, 0.0078125)


def quantize(x, fmt):
    """Codes and scale bytes by the layer's rule, in float64."""
    T, H = x.shape
    if fmt == "per_tensor":
        q = (x.double() / SCALES[0]).clamp(-448, 448)
        return q.float().to(torch.float8_e4m3fn).view(torch.uint8), None
    b = {"deepseek": 128, "mxfp8": 32}[fmt]
    v = x.double().view(T, -1, b)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax / 448)
    e = torch.where(m == 0.5, e - 1, e)            # least 2^e >= amax / 448
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-127, 127)
    q = v * torch.exp2(-e.double())[..., None]
    q = q.float().to(torch.float8_e4m3fn).view(torch.uint8).view(T, H)
    return q, (e + 127).to(torch.uint8)


def values(q, s, fmt):
    v = q.view(torch.float8_e4m3fn).double()
    if s is None:
        return v * SCALES[0]
    b = v.shape[1] // s.shape[1]
    return (v.view(v.shape[0], -1, b) * torch.exp2(s.double() - 127)[..., None]).view_as(v)


@pytest.mark.parametrize("fmt", ["deepseek", "mxfp8", "per_tensor"])
@pytest.mark.parametrize("T,H,I,E,K", [(1, 256, 128, 4, 1), (7, 384, 256, 8, 2), (40, 512, 256, 8, 4),
                                       (333, 640, 384, 8, 6), (1100, 256, 128, 16, 8)])
def test_same_bits_as_from_bf16(S, orc, fmt, T, H, I, E, K):
    x, idx, w, w1, w2 = small_problem(orc, T, H, I, E, K, seed=T + H)
    xt, it, wt = gh.to_device(x, idx, w)
    xt[T // 2, :128] = 0
    if K > 1:
        it[0, 1] = -1
    m = layer(S, H, I, E, K, T, fmt, w1, w2)
    want = m.forward(xt, it, wt).clone()
    assert m.read_status() == (0, 0)
    q, s = quantize(xt, fmt)
    got = m.forward_quantized(q, s, it, wt)
    assert m.read_status() == (0, 0)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", ["deepseek", "mxfp8", "per_tensor"])
@pytest.mark.parametrize("fused", [False, True])
def test_norm_route_and_layer_in_eight_bits(S, orc, fmt, fused):
    """norm -> route -> layer as a block runs them, in a graph."""
    T, H, I, E, K = 77, 512, 256, 16, 4
    x, _, _, w1, w2 = small_problem(orc, T, H, I, E, K, seed=5)
    xt = torch.from_numpy(x.view(np.int16).copy()).cuda().view(torch.bfloat16)
    gen = torch.Generator("cuda").manual_seed(6)
    res = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    gain = (torch.rand(H, device="cuda", generator=gen) + 0.5).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=gen)
    m = layer(S, H, I, E, K, T, fmt, w1, w2, fuse_fc1=fused)

    def block():
        _, r, q, s = S.add_rms_norm(xt, gain, residual=res, fmt=fmt, scale=SCALES[0])
        idx, w = S.topk_route(logits, K)
        return r, q, s, idx, w, m.forward_quantized(q, s, idx, w)

    r, q, s, idx, w, got = block()
    got = got.clone()
    assert m.read_status() == (0, 0)
    v = values(q, s, fmt).bfloat16()
    assert torch.equal(v.double(), values(q, s, fmt))
    # (a block whose largest code rounded down to half of the range gets the next smaller
    # scale there: the same values, other products inside the matrix unit)
    ref = m.forward(v, idx, w).double()
    assert (got.double() - ref).norm() <= 1e-2 * ref.norm()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block()
    res.neg_()
    g.replay()
    torch.cuda.synchronize()
    again = block()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out[:5], again[:5]) if a is not None)
    assert not torch.equal(out[0], r)


def test_refusals(S, orc):
    B = S.binding
    T, H, I, E, K = 9, 256, 128, 4, 2
    x, idx, w, w1, w2 = small_problem(orc, T, H, I, E, K, seed=2)
    xt, it, wt = gh.to_device(x, idx, w)
    m = layer(S, H, I, E, K, T, "deepseek", w1, w2)
    q, s = quantize(xt, "deepseek")
    st = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()
    for args, status in (((0, p(s), p(it), p(wt), T), B.MOE_ERR_INVALID_ARG),
                         ((p(q), 0, p(it), p(wt), T), B.MOE_ERR_INVALID_ARG),
                         ((p(q), p(s), 0, p(wt), T), B.MOE_ERR_INVALID_ARG),
                         ((p(q), p(s), p(it), 0, T), B.MOE_ERR_INVALID_ARG),
                         ((p(q) + 8, p(s), p(it), p(wt), T), B.MOE_ERR_INVALID_ARG),
                         ((p(q), p(s), p(it), p(wt), -1), B.MOE_ERR_INVALID_ARG),
                         ((p(q), p(s), p(it), p(wt), T + 1), B.MOE_ERR_CAPACITY)):
        with pytest.raises(B.MoEError) as e:
            B.moe_forward_quantized(m.handle, *args, st)
        assert e.value.status == status
    assert m.forward_quantized(q[:0], s[:0], it[:0], wt[:0]).shape == (0, H)
    for bad in ((q, s[:, :1], it, wt), (q, None, it, wt), (q[:, :128], s, it, wt), (xt, s, it, wt)):
        with pytest.raises((AssertionError, AttributeError)):
            m.forward_quantized(*bad)
    fresh = S.MegaMoELayer(H, I, E, K, max_rows=T)
    with pytest.raises(B.MoEError) as e:
        B.moe_forward_quantized(fresh.handle, p(q), p(s), p(it), p(wt), T, st)
    assert e.value.status == B.MOE_ERR_NOT_BOUND
