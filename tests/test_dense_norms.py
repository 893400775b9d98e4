"""The bounds that the GPU tests hold the dense products to, against products with planted
mistakes (no GPU needed): a bound in norm sees what the elementwise worst case of a long row lets pass."""
import torch

from tests import dense_norms as norms
from tests import dense_reference as ref


def planted(K, what):
    g = torch.Generator().manual_seed(K)
    a, b = (torch.randn(n, K, generator=g).bfloat16().double() for n in (16, 130))
    want, tol = ref.product(a, b)
    if what == "columns":
        got = a[:, :-16] @ b[:, :-16].t()
    elif what == "block":
        got = a[:, 128:] @ b[:, 128:].t()
    else:  # sums kept in BF16
        got = torch.zeros_like(want)
        for k in range(0, K, 128):
            got = (got + a[:, k:k + 128] @ b[:, k:k + 128].t()).bfloat16().double()
    return want, got, tol


def test_long_rows():
    for K in (7168, 32768):
        for what in ("columns", "block", "bf16"):
            want, got, _ = planted(K, what)
            err = float((got - want).norm() / want.norm())
            assert err > 4 * norms.summed(K), (K, what, err, norms.summed(K))
            if what != "bf16":  # a lost column shows in rounded outputs too
                assert err > norms.rounded(torch.bfloat16)
    want, got, tol = planted(32768, "bf16")
    assert ((got - want).abs() <= tol).all()  # (which the elementwise bound alone would pass)


def test_sums_in_float_stay_within():
    """Steps of 32 products truncated to 24 bits, the worst the bound is made for."""
    K, g = 7168, torch.Generator().manual_seed(1)
    a, b = (torch.randn(n, K, generator=g).bfloat16().double() for n in (16, 130))
    s = torch.zeros(16, 130, dtype=torch.float64)
    for k in range(0, K, 32):
        s = s + a[:, k:k + 32] @ b[:, k:k + 32].t()
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.trunc(torch.ldexp(m, torch.tensor(24))), e - 24)
    want = a @ b.t()
    assert float((s - want).norm() / want.norm()) <= norms.summed(K)
