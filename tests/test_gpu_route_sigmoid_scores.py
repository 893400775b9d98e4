"""GPU: the sigmoid scores of moe_topk_route are those of the float formula, 1 / (1 + exp(-l))
with a correctly rounded sum and quotient.
"""
import pytest
import torch

from tests.test_gpu_decode_fp4 import S  # noqa: F401

pytestmark = pytest.mark.gpu


def test_scores_below_the_normal_numbers(S):  # noqa: F811
    """exp(-l) is finite up to 88.72, and from 87.34 on the score is a subnormal number,
    at least 3.3e-39 here: 2^-22 relative by its last bit, 2^-22 by exp, 2^-23 by the sum and the quotient;
    twice that, and 2^-23, for a share of their sum."""
    gen = torch.Generator("cuda").manual_seed(1)
    l = -87.4 - 1.2 * torch.rand(50, 64, device="cuda", generator=gen)
    idx, w = S.topk_route(l, 4, scoring="sigmoid", scale=2.5)
    p = torch.sigmoid(l.double()).gather(1, idx.long())
    want = 2.5 * p / p.sum(-1, keepdim=True)
    assert torch.all((w.double() - want).abs() <= 2.0**-20 * want)
    idx, w = S.topk_route(l, 4, scoring="sigmoid", renormalize=False)
    assert torch.all((w.double() - p).abs() <= 2.0**-22 * p + 2.0**-149) and torch.all(w > 0)


@pytest.mark.parametrize("G,TG", [(1, 1), (8, 4)])
@pytest.mark.parametrize("biased", [False, True])
def test_choices_of_the_float_formula(S, G, TG, biased):  # noqa: F811
    """Scores one unit in the last place apart are in the right order: the ids are those of
    a stable sort of the float formula's values, equal ones by their index."""
    T, E, K = 8192, 256, 8
    gen = torch.Generator("cuda").manual_seed(2)
    bias = 0.05 * torch.randn(E, device="cuda", generator=gen) if biased else None
    wrong = 0
    for _ in range(8):
        l = torch.randn(T, E, device="cuda", generator=gen)
        idx, _ = S.topk_route(l, K, scoring="sigmoid", bias=bias, num_groups=G, top_groups=TG)
        c = 1.0 / (1.0 + torch.exp(-l))
        if biased:
            c = c + bias
        if G > 1:
            by = c.view(T, G, -1)
            best = by.sort(dim=-1, descending=True)[0][..., :2].sum(-1)
            keep = best.sort(dim=-1, descending=True, stable=True)[1][:, :TG]
            mask = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, keep, True)
            c = torch.where(mask[..., None], by, -torch.inf).view(T, E)
        want = c.sort(dim=-1, descending=True, stable=True)[1][:, :K]
        wrong += int((idx != want).any(-1).sum())
    assert wrong == 0
