"""Making a handle on one stream and using it on another."""
import pytest
import torch

from tests.test_gpu_dense import BF, S, mlp_case, rand, weights8  # noqa: F401

pytestmark = pytest.mark.gpu


def busy_stream():
    """A stream that has 50 ms or so before it."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    return side


def workspace(n):
    w = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # what memory may hold
    torch.cuda.synchronize()
    return w


def test_mlp_made_on_a_busy_stream(S):
    """A handle is ready for any stream when its creation returns."""
    B = S.binding
    w1, w2, x, mlp = mlp_case(S, 8, 264, 136, BF, "silu")
    want = mlp.forward(x)
    n = B.moe_mlp_workspace_query(264, 136, 8)
    ws = workspace(n)
    side = busy_stream()
    h = B.moe_mlp_create(264, 136, 0, B.MOE_ACT_SILU, 0, 8, w1.data_ptr(), w2.data_ptr(), ws.data_ptr(), n,
                         side.cuda_stream)
    main = torch.cuda.current_stream().cuda_stream
    assert B.moe_mlp_read_status(h, main) == (B.MOE_OK, 0)
    y = torch.empty_like(want)
    B.moe_mlp_forward(h, x.data_ptr(), 264, 8, y.data_ptr(), 0, 0, main)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and B.moe_mlp_read_status(h, main) == (B.MOE_OK, 0)
    B.moe_mlp_destroy(h)


def test_linear_made_on_a_busy_stream(S):
    B = S.binding
    codes, scales = weights8(200, 256)
    x = rand(8, 256, seed=1)
    want = S.Fp8Linear(codes, scales, max_tokens=8).forward(x)
    n = B.moe_fp8_linear_workspace_query(200, 256, 8)
    ws = workspace(n)
    side = busy_stream()
    h = B.moe_fp8_linear_create(200, 256, 0, 8, codes.data_ptr(), scales.data_ptr(), ws.data_ptr(), n, side.cuda_stream)
    main = torch.cuda.current_stream().cuda_stream
    y = torch.empty_like(want)
    B.moe_fp8_linear(h, x.data_ptr(), 256, 8, y.data_ptr(), 0, main)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and B.moe_fp8_linear_read_status(h, main) == (B.MOE_OK, 0)
    B.moe_fp8_linear_destroy(h)
