"""The bounded waits of the NVFP4 layer's kernel, without a GPU fault.

With MOE_FLAG_WATCHDOG_TEST the first CTA's first copying warp asks for
nothing and the limit is 20 ms: the consumers there wait for copies that never
begin, the other CTAs at the grid barrier for h that never comes.  All must
give up, record MOE_DEV_TIMEOUT and return, the counters must be at zero for
the next call, and the context usable.
"""
import pytest
import torch

from tests.test_gpu_decode_fp4 import S, check_layer, fp4, routes  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 11])
def test_waits_expire_with_status_and_context_survives(S, T):  # noqa: F811
    B = S.binding
    H, I, E, K = 1024, 512, 16, 4
    gen = torch.Generator("cuda").manual_seed(31)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    idx, w = routes(gen, T, E, K)
    bad = S.Fp4MoELayer(H, I, E, K, watchdog_test=True)
    bad.bind_weights(*p1, *p2)
    for _ in range(2):  # the first leaves nothing behind that the second one trips over
        bad.forward(x, idx, w)
        assert bad.read_status() == (B.MOE_ERR_DEVICE_TIMEOUT, B.MOE_DEV_TIMEOUT)
    check_layer(S, p1, p2, x, idx, w)
    # the same workspace, on a handle that withholds nothing
    good = S.Fp4MoELayer(H, I, E, K)
    want, _ = check_layer(S, p1, p2, x, idx, w)
    good.weights, good.workspace = bad.weights, bad.workspace
    good.handle = B.moe_fp4_create(H, I, E, K, good.flags, 16, *(t.data_ptr() for t in good.weights),
                                   good.workspace.data_ptr(), good._ws_bytes,
                                   torch.cuda.current_stream().cuda_stream)
    assert torch.equal(good.forward(x, idx, w), want) and good.read_status() == (0, 0)


def test_a_timeout_is_reported_until_it_is_read(S):  # noqa: F811
    """Calls after one that gave up, on the same workspace, say so too, until the
    status has been read; then they are normal."""
    B = S.binding
    H, I, E, K, T = 1024, 512, 16, 4, 3
    gen = torch.Generator("cuda").manual_seed(33)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    idx, w = routes(gen, T, E, K)
    want, good = check_layer(S, p1, p2, x, idx, w)
    bad = S.Fp4MoELayer(H, I, E, K, watchdog_test=True)
    bad.weights, bad.workspace = good.weights, good.workspace
    bad.handle = B.moe_fp4_create(H, I, E, K, bad.flags, 16, *(t.data_ptr() for t in bad.weights),
                                  bad.workspace.data_ptr(), bad._ws_bytes, torch.cuda.current_stream().cuda_stream)
    bad.forward(x, idx, w)
    good.forward(x, idx, w)
    assert good.read_status() == (B.MOE_ERR_DEVICE_TIMEOUT, B.MOE_DEV_TIMEOUT)
    for _ in range(2):
        assert torch.equal(good.forward(x, idx, w), want) and good.read_status() == (0, 0)
