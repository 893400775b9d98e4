"""GPU: moe_fp4_linear at the widest and the tallest matrices that it takes.

Wide rows leave room for few tokens at a time, down to one, so that sixteen tokens sweep the
matrix up to sixteen times; 2^24 rows of 32 columns are 2^19 tiles.
"""
import pytest
import torch

from tests.test_gpu_decode_fp4 import S, check_linear, fp4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [7168, 16416, 20000, 24576, 32736, 32768])
@pytest.mark.parametrize("rows", [40, 5000])
def test_wide(S, rows, cols):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(cols)
    c, s, g = fp4(gen, 1, rows, cols)
    parts = (c[0], s[0], g)
    lin = S.Fp4Linear(*parts)
    for T in (1, 2, 5, 12, 13, 16):
        x = torch.randn(T, cols, device="cuda", generator=gen).bfloat16()
        check_linear(S, lin, parts, x, True)


@pytest.mark.parametrize("rows", [100003, (1 << 24) - 1, 1 << 24])
def test_tall(S, rows):  # noqa: F811
    """Sums that are exact: codes of 1, x of powers of two, scales that are multiples of 1/8."""
    cols = 32
    codes = torch.full((rows, cols // 2), 0x22, dtype=torch.uint8, device="cuda")
    gen = torch.Generator("cuda").manual_seed(rows)
    scales = torch.randint(0x38, 0x70, (rows, cols // 16), dtype=torch.uint8, device="cuda", generator=gen)
    lin = S.Fp4Linear(codes, scales, torch.ones(1, device="cuda"))
    want = 16 * scales.view(torch.float8_e4m3fn).float().sum(-1)
    for T in (1, 3, 16):
        up = torch.exp2(torch.arange(T, device="cuda") % 5)
        y = lin.forward(up[:, None].expand(T, cols).bfloat16(), out_dtype=torch.float32)
        for t in range(T):
            assert torch.equal(y[t], want * up[t])
    assert lin.read_status() == (0, 0)
