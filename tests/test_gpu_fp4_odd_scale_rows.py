"""moe_fp4_linear where a row's scales are an odd multiple of two bytes (columns
that are odd multiples of 32): they reach shared memory by ordinary stores, so
the signal that they are there has to order ordinary stores.
"""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_stored_scales_are_released():
    """No GPU shows a missing order reliably, so the source is looked at: what follows
    the stores of the scales is an arrival that releases them, not one that is triggered by
    asynchronous copies."""
    with open(os.path.join(ROOT, "serving_route_gb300", "csrc", "fp4.cu")) as f:
        src = f.read()
    producer = src[src.index("-- producers"):src.index("-- epilogue")]
    stores = [m.end() for m in re.finditer(r"st\.shared", producer)]
    assert stores
    for at in stores:
        arrival = re.search(r"mbar_arrive\(bar\)|cp\.async\.mbarrier\.arrive", producer[at:])
        assert arrival and arrival.group() == "mbar_arrive(bar)"


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(40001, 4064), (20000, 544), (9000, 7200)])
def test_no_scale_of_the_lap_before(rows, cols):
    """Every place of the ring is used several times, with other scales each time, and all
    sums are exact: codes and x are 1, the scales multiples of 1/8 below 512, so that a
    sum of at most 450 of them, 16 times each, is below 2^24 / 8."""
    import __graft_entry__ as ge
    ge.build()
    import serving_route_gb300 as S
    gen = torch.Generator("cuda").manual_seed(rows)
    codes = torch.full((rows, cols // 2), 0x22, dtype=torch.uint8, device="cuda")
    scales = torch.randint(0x38, 0x70, (rows, cols // 16), dtype=torch.uint8, device="cuda", generator=gen)
    lin = S.Fp4Linear(codes, scales, torch.ones(1, device="cuda"))
    want = 16 * scales.view(torch.float8_e4m3fn).double().sum(-1)
    assert want.max() < 2**21
    for T in (1, 9):
        x = torch.ones(T, cols, dtype=torch.bfloat16, device="cuda")
        for _ in range(10):
            y = lin.forward(x, out_dtype=torch.float32)
            assert torch.equal(y.double(), want.expand(T, -1))
    assert lin.read_status() == (0, 0)
