"""GPU: norm -> route -> forward_quantized on a side stream and in a graph gives the layer's
output of the same calls one by one, bit for bit, for inputs that change between replays.

The norm's launch overlaps what is before it and the dispatch reads its codes: a wait that
is missing between the two shows as codes of the inputs before.
"""
import pytest
import torch

from tests import gpu_harness as gh
from tests.test_gpu_parity import small_problem
from tests.test_gpu_quantized_rows import S, SCALES, layer  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["deepseek", "mxfp8", "per_tensor"])
@pytest.mark.parametrize("T,fused", [(5, False), (77, True), (1500, True)])
def test_outputs(S, orc, fmt, T, fused):  # noqa: F811
    H, I, E, K = 512, 256, 16, 4
    x, idx0, w0, w1, w2 = small_problem(orc, T, H, I, E, K, seed=T)
    xt = gh.to_device(x, idx0, w0)[0]
    gen = torch.Generator("cuda").manual_seed(T)
    res = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    gain = (torch.rand(H, device="cuda", generator=gen) + 0.5).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=gen)
    m = layer(S, H, I, E, K, T, fmt, w1, w2, fuse_fc1=fused)

    def block():
        _, r, q, s = S.add_rms_norm(xt, gain, residual=res, fmt=fmt, scale=SCALES[0])
        return (r, q, s, *S.topk_route(logits, K)), lambda i, w: m.forward_quantized(q, s, i, w)

    def whole():
        made, forward = block()
        return made, forward(*made[3:])

    def one_by_one():
        made, forward = block()
        torch.cuda.synchronize()
        out = forward(*made[3:])
        torch.cuda.synchronize()
        assert m.read_status() == (0, 0)
        return [None if t is None else t.clone() for t in made], out.clone()

    def new_inputs():
        res.copy_(torch.randn(T, H, device="cuda", generator=gen))
        logits.copy_(torch.randn(T, E, device="cuda", generator=gen))

    def same(got, want):
        return all(torch.equal(a, b) for a, b in zip(got, want) if b is not None)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made, out = whole()
    last = None
    for _ in range(4):
        new_inputs()
        want, want_out = one_by_one()
        assert last is None or not torch.equal(want_out, last)
        last = want_out
        m.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(made, want) and torch.equal(out, want_out)
        m.out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            side_made, side_out = whole()
        side.synchronize()
        assert same(side_made, want) and torch.equal(side_out, want_out)
        assert m.read_status() == (0, 0)
