"""GPU: moe_topk_route with many equal logits, against a stable descending sort.

Logits from a few values (multiples of 1/4, exact in BF16): equal ones must be
chosen by their index, whichever lane or row of the warp holds them, in every
number of choices; sigmoid is strictly monotone at this spacing, and equal
logits give equal scores.  Ids must be equal exactly; weights by the formula in
float64 within 2e-6 relative (float exp and sums).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    import __graft_entry__ as ge
    ge.build()
    import serving_route_gb300
    return serving_route_gb300


@pytest.mark.parametrize("E", [8, 32, 40, 64, 128, 160, 256, 512, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ties(S, E, dtype, scoring):
    gen = torch.Generator("cuda").manual_seed(E)
    for levels in (1, 3, 17):
        x = torch.randint(0, levels, (65, E), device="cuda", generator=gen).float() / 4 - 1
        x[7, E // 2:] = -torch.inf                   # fewer experts left than choices, for a small E
        x[9] = -torch.inf
        x = x.to(dtype)
        for K in sorted({1, 2, min(6, E), min(8, E), min(32, E)}):
            idx, w = S.topk_route(x, K, scoring=scoring)
            order = torch.sort(x.double(), dim=-1, descending=True, stable=True)
            want = torch.where(order.values[:, :K] > -torch.inf, order.indices[:, :K], -1)
            assert torch.equal(idx.long(), want)
            d = x.double()
            p = torch.sigmoid(d) if scoring == "sigmoid" else torch.softmax(d, -1).nan_to_num(0.0)
            p = torch.where(want >= 0, p.gather(1, want.clamp(min=0)), 0.0)
            s = p.sum(-1, keepdim=True)
            p = torch.where(s > 0, p / s, 0.0)
            assert torch.all((w.double() - p).abs() <= 2e-6 * p)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,top", [(256, 8, 4), (64, 2, 1), (160, 8, 3), (512, 16, 5)])
def test_tied_groups(S, E, groups, top, dtype):
    """Groups of equal score: the lowest ones are kept."""
    gen = torch.Generator("cuda").manual_seed(E + groups)
    x = (torch.randint(0, 4, (65, E), device="cuda", generator=gen).float() / 4).to(dtype)
    K = 6
    idx, _ = S.topk_route(x, K, num_groups=groups, top_groups=top)
    d = x.double().view(65, groups, -1)
    best = torch.sort(d.amax(-1), dim=-1, descending=True, stable=True).indices[:, :top]
    keep = torch.zeros(65, groups, dtype=torch.bool, device="cuda").scatter_(1, best, True)
    d = torch.where(keep[..., None], d, -torch.inf).view(65, E)
    assert torch.equal(idx.long(), torch.sort(d, dim=-1, descending=True, stable=True).indices[:, :K])
