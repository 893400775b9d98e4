"""GPU: rows of gate logits without a number reach the forwards' route checks.

A NaN hidden state makes every logit of its token NaN.  No expert can be chosen
there, and the forwards skip slots of id -1; so such a row has to name an expert beside its
NaN weight, or the layer would answer zeros and report nothing.
"""
import math

import pytest
import torch

from tests import gpu_harness as gh
from tests.test_gpu_decode_fp4 import S, fp4  # noqa: F401
from tests.test_gpu_parity import small_problem

pytestmark = pytest.mark.gpu
NAN, INF = math.nan, math.inf


@pytest.mark.parametrize("E,G,TG", [(1, 1, 1), (8, 1, 1), (40, 1, 1), (64, 4, 2), (256, 8, 4), (160, 8, 3), (1000, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_a_row_with_a_nan_names_an_expert(S, E, G, TG, dtype, scoring):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(E)
    l = torch.randn(9, E, device="cuda", generator=gen)
    l[8] = -INF                        # masked, which is not NaN
    good = [0, 3, 7, 8]
    at = {1: 0, 2: E - 1, 4: E // 2, 5: 0, 6: 0}
    l[1] = NAN
    l[2], l[2, E - 1] = -INF, NAN      # masked but for the last, which is NaN
    l[4], l[4, E // 2] = -INF, NAN
    l[5] = -NAN                        # the other sign
    l[6] = NAN
    l[6, 1:3] = 1.0                    # fewer numbers than choices
    l = l.to(dtype)
    for K in sorted({1, min(4, E), min(8, E)}):
        idx, w = S.topk_route(l, K, scoring=scoring, num_groups=G, top_groups=TG)
        ref = S.topk_route(l[good], K, scoring=scoring, num_groups=G, top_groups=TG)
        assert torch.equal(idx[good], ref[0]) and torch.equal(w[good], ref[1]) and torch.isfinite(w[good]).all()
        for t, first in at.items():
            assert torch.isnan(w[t]).all()
            if t == 6 and E > 1:       # numbers go before
                n = min(K, 2)
                assert idx[t, :n].tolist() == [1, 2][:n] and torch.all(idx[t, n:] == -1)
            else:                      # the lowest expert that holds a NaN
                assert idx[t].tolist() == [first] + [-1] * (K - 1)
        assert torch.all(idx[8] == -1) and not w[8].any()


def test_a_nan_bias_names_an_expert(S):  # noqa: F811
    E, K = 48, 4
    l = torch.randn(3, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    l[1, :5] = -INF
    bias = torch.full((E,), NAN, device="cuda")
    idx, w = S.topk_route(l, K, scoring="sigmoid", bias=bias)
    assert torch.isnan(w).all() and torch.all(idx[:, 0] == 0) and torch.all(idx[:, 1:] == -1)
    bias[:10] = -INF
    idx, w = S.topk_route(l, K, scoring="sigmoid", bias=bias)
    assert torch.isnan(w).all() and torch.all(idx[:, 0] == 10) and torch.all(idx[:, 1:] == -1)


def nan_routes(S, T, E, K, bad, **kw):  # noqa: F811
    l = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(E))
    bad(l)
    return S.topk_route(l, K, **kw)


BAD = [lambda l: l[2].fill_(NAN), lambda l: l[2, 1:].fill_(NAN), lambda l: l.fill_(NAN),
       lambda l: (l[2].fill_(-INF), l[2, 5:6].fill_(NAN))]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_the_few_token_layer_reports_them(S, bad, scoring):  # noqa: F811
    B, (T, H, I, E, K) = S.binding, (4, 256, 128, 8, 2)
    gen = torch.Generator("cuda").manual_seed(2)
    layer = S.Fp4MoELayer(H, I, E, K)
    layer.bind_weights(*fp4(gen, E, 2 * I, H), *fp4(gen, E, H, I))
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    idx, w = nan_routes(S, T, E, K, bad, scoring=scoring)
    layer.forward(x, idx, w)
    assert layer.read_status() == (B.MOE_ERR_BAD_ROUTE, B.MOE_DEV_ROUTE_NONFINITE)
    layer.forward(x, *nan_routes(S, T, E, K, lambda l: l[2].fill_(-INF), scoring=scoring))
    assert layer.read_status() == (0, 0)
    free = S.Fp4MoELayer(H, I, E, K, check_routes=False)
    free.bind_weights(*layer.weights)
    assert torch.isnan(free.forward(x, idx, w)[2]).all()  # unchecked, the token is NaN, not zero


@pytest.mark.parametrize("bad", BAD)
def test_the_fp8_layer_reports_them(S, orc, bad):  # noqa: F811
    B, (T, H, I, E, K) = S.binding, (4, 256, 128, 8, 2)
    x, _, _, w1, w2 = small_problem(orc, T, H, I, E, K, seed=3)
    xt = gh.to_device(x, torch.zeros(1).numpy(), torch.zeros(1).numpy())[0]
    q1, s1 = S.MegaMoELayer.quantize_weights(torch.from_numpy(w1).cuda())
    q2, s2 = S.MegaMoELayer.quantize_weights(torch.from_numpy(w2).cuda())
    m = S.MegaMoELayer(H, I, E, K, max_rows=T)
    m.bind_weights(q1, s1, q2, s2)
    m.forward(xt, *nan_routes(S, T, E, K, bad))
    assert m.read_status() == (B.MOE_ERR_BAD_ROUTE, B.MOE_DEV_ROUTE_NONFINITE)
    m.forward(xt, *nan_routes(S, T, E, K, lambda l: l[2].fill_(-INF)))
    assert m.read_status() == (0, 0)
