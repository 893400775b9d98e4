"""The block's gradients of no rows: zeros in the weights' gradients, and the same refusals as of some."""
import pytest
import torch

from tests.test_gpu_dense import BF, S, mlp_case  # noqa: F401
from tests.test_gpu_dense_edges import status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [0, 1])
def test_gradients_of_no_rows_over_the_weights(S, accumulate):
    B = S.binding
    w1, w2, _, mlp = mlp_case(S, 8, 64, 32, BF, "silu", seed=5)
    kept = w1.clone(), w2.clone()
    free = torch.ones(2, 64, 64, device="cuda")
    a, b = free[0].data_ptr(), free[1].data_ptr()

    def call(dw1, dw2):
        return status(B, B.moe_mlp_backward, mlp.handle, 0, 64, 0, 64, 0, 1, 0, 0, dw1, dw2, 1, accumulate, 0)

    for dw1, dw2 in ((w1.data_ptr(), 0), (0, w1.data_ptr()), (w2.data_ptr(), b), (a, w2.data_ptr()), (a, a),
                     (a, a + 64 * 64 * 4 - 16)):
        assert call(dw1, dw2) == B.MOE_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(w1, kept[0]) and torch.equal(w2, kept[1]) and (free == 1).all()
    assert call(a, b) == B.MOE_OK
    assert (free[0] == accumulate).all() and (free[1].view(-1)[:64 * 32] == accumulate).all()
    assert (free[1].view(-1)[64 * 32:] == 1).all()
