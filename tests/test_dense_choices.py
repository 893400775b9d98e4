"""The sizes the GPU tests use reach every kernel of the dense products (no GPU needed), and
plans of no handle are refused."""
import ctypes

import pytest

from tests import dense_choices as c


@pytest.fixture(scope="module")
def B():
    from serving_route_gb300 import build
    build.build()
    import serving_route_gb300.binding as B
    return B


@pytest.mark.parametrize("launch", c.LAUNCHES)
def test_block_sizes_reach_every_choice(launch):
    seen = {row[3 + c.LAUNCHES.index(launch)] for row in c.MLP}
    want = {(c.P, w) for w in (64, 128, 192, 256)}
    if launch != "gradients":  # (that launch is the pairs' alone)
        want |= {(c.K, s) for s in (1, 2, 4, 8)}
    assert {s for s in seen if s[0] == c.P} >= {s for s in want if s[0] == c.P}
    # the split kernel's three forms differ in what they finish: together they see every share
    assert launch == "gradients" or len({s for s in seen if s[0] == c.K}) >= 3


def test_linear_sizes_reach_every_choice():
    seen = {row[3] for row in c.LINEAR}
    assert seen == {(c.P, w) for w in (64, 128, 192, 256)} | {(c.K, s) for s in (1, 2, 4, 8)}


def test_plans_of_nothing(B):
    L, p = B.lib(), (B.moe_dense_launch * 4)()
    assert L.moe_fp8_linear_plan(None, 1, 0, p) == B.MOE_ERR_INVALID_ARG
    assert L.moe_mlp_plan(None, 1, p) == B.MOE_ERR_INVALID_ARG


def test_flags_of_the_block(B):
    A = 0x7000000000  # an address, not memory: refused before anything reads it
    for flags in (B.MOE_FLAG_WATCHDOG_LAST_TEST << 1, B.MOE_FLAG_WATCHDOG_LAST_TEST | 1):
        with pytest.raises(B.MoEError) as e:
            B.moe_mlp_create(64, 32, 0, 0, flags, 4, A, A, A, 1 << 20, 0)
        assert e.value.status == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(B.MoEError) as e:
        B.moe_fp8_linear_create(64, 256, B.MOE_FLAG_WATCHDOG_LAST_TEST, 4, A, A, A, 1 << 20, 0)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
