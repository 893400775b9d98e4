"""Host-side checks of the few-token operators (no GPU needed): what the calls
refuse they refuse before any CUDA call, and the workspace queries apply the
documented rules.  The addresses below are numbers, not memory: no call here
reads them."""
import ctypes

import pytest

A = 0x7000000000  # a 16-byte aligned "device address"


@pytest.fixture(scope="module")
def B():
    from serving_route_gb300 import build
    build.build()
    import serving_route_gb300.binding as B
    return B


def status(B, call, *args):
    try:
        call(*args)
    except B.MoEError as e:
        return e.status
    return B.MOE_OK


NORM = dict(x=A, x_stride=256, residual=0, residual_stride=0, weight=A, eps=1e-6, num_tokens=4, hidden=256,
            residual_out=0, y=A, q=0, q_scale=0, q_format=0, q_static_scale=1.0, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(x=0), "INVALID_ARG"), (dict(weight=0), "INVALID_ARG"), (dict(y=0), "INVALID_ARG"),
    (dict(x=A + 1), "INVALID_ARG"), (dict(y=A + 1), "INVALID_ARG"), (dict(weight=A + 1), "INVALID_ARG"),
    (dict(x_stride=255), "INVALID_ARG"), (dict(num_tokens=-1), "INVALID_ARG"), (dict(hidden=0), "INVALID_ARG"),
    (dict(eps=-1e-6), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(residual=A, residual_stride=256), "INVALID_ARG"),              # r has nowhere to go
    (dict(residual_out=A), "INVALID_ARG"),                               # there is no r
    (dict(residual=A, residual_stride=255, residual_out=A), "INVALID_ARG"),
    (dict(x_stride=300), "INVALID_ARG"),                                 # y in place of strided rows
    (dict(q=A), "INVALID_ARG"),                                          # no scales
    (dict(q=A, q_format="PER_TENSOR", q_static_scale=0.0), "INVALID_ARG"),
    (dict(q=A, q_format="PER_TENSOR", q_static_scale=float("nan")), "INVALID_ARG"),
    (dict(q=A, q_format="PER_TENSOR", q_static_scale=float("inf")), "INVALID_ARG"),
    (dict(hidden=192, x_stride=192, q=A, q_scale=A), "UNSUPPORTED"),
    (dict(hidden=176, x_stride=176, q=A, q_scale=A, q_format="MXFP8"), "UNSUPPORTED"),
    (dict(hidden=(1 << 20) + 8, x_stride=1 << 21), "UNSUPPORTED"),
    (dict(num_tokens=0), "OK"), (dict(num_tokens=0, x=0, weight=0, y=0), "OK"),
])
def test_norm(B, change, want):
    kw = {**NORM, **change}
    if isinstance(kw["q_format"], str):
        kw["q_format"] = getattr(B, "MOE_FLAG_" + kw["q_format"])
    assert status(B, B.moe_add_rms_norm, *kw.values()) == getattr(B, "MOE_OK" if want == "OK" else "MOE_ERR_" + want)


ROUTE = dict(logits=A, bf16=0, stride=64, bias=0, num_tokens=4, num_experts=64, top_k=4, sigmoid=0, num_groups=1,
             top_groups=1, renormalize=1, scale=1.0, idx=A, w=A, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(logits=0), "INVALID_ARG"), (dict(idx=0), "INVALID_ARG"), (dict(w=0), "INVALID_ARG"),
    (dict(stride=63), "INVALID_ARG"), (dict(num_tokens=-1), "INVALID_ARG"),
    (dict(logits=A + 2), "INVALID_ARG"), (dict(logits=A + 1, bf16=1), "INVALID_ARG"),
    (dict(idx=A + 2), "INVALID_ARG"), (dict(w=A + 2), "INVALID_ARG"),
    (dict(num_experts=0, stride=0), "UNSUPPORTED"), (dict(num_experts=1025, stride=1025), "UNSUPPORTED"),
    (dict(top_k=0), "UNSUPPORTED"), (dict(top_k=33), "UNSUPPORTED"),
    (dict(num_experts=3, stride=3, top_k=4), "UNSUPPORTED"),
    (dict(num_groups=0), "UNSUPPORTED"), (dict(num_groups=7), "UNSUPPORTED"),
    (dict(num_groups=64, top_groups=2), "UNSUPPORTED"), (dict(num_groups=8, top_groups=9), "UNSUPPORTED"),
    (dict(num_groups=8, top_groups=0), "UNSUPPORTED"), (dict(bias=A), "UNSUPPORTED"),
    (dict(num_tokens=0), "OK"), (dict(num_tokens=0, logits=0, idx=0, w=0), "OK"),
])
def test_route(B, change, want):
    kw = {**ROUTE, **change}
    assert status(B, B.moe_topk_route, *kw.values()) == getattr(B, "MOE_OK" if want == "OK" else "MOE_ERR_" + want)


@pytest.mark.parametrize("dims,flags,tokens,want", [
    ((7168, 2048, 256, 8), 0, 16, "OK"), ((128, 128, 1, 1), 2, 1, "OK"), ((16384, 16384, 1024, 6), 0, 16, "OK"),
    ((192, 128, 4, 1), 0, 1, "UNSUPPORTED"), ((128, 64, 4, 1), 0, 1, "UNSUPPORTED"),
    ((16512, 128, 4, 1), 0, 1, "UNSUPPORTED"), ((128, 128, 0, 1), 0, 1, "UNSUPPORTED"),
    ((128, 128, 1025, 1), 0, 1, "UNSUPPORTED"), ((128, 128, 4, 3), 0, 1, "UNSUPPORTED"),
    ((128, 128, 4, 2), 0x1, 1, "UNSUPPORTED"), ((128, 128, 4, 2), 0x100, 1, "UNSUPPORTED"),
    ((128, 128, 4, 2), 0, 17, "UNSUPPORTED"), ((128, 128, 4, 2), 0, 0, "INVALID_ARG"),
])
def test_layer_query(B, dims, flags, tokens, want):
    want = B.MOE_OK if want == "OK" else getattr(B, "MOE_ERR_" + want)
    assert status(B, B.moe_fp4_workspace_query, *dims, flags, tokens) == want
    if want == B.MOE_OK:  # h in half, an exponent per 16 values, for every route
        n = [B.moe_fp4_workspace_query(*dims, flags, t) for t in (1, tokens)]
        assert n[1] - n[0] >= (tokens - 1) * dims[3] * (2 * dims[1] + dims[1] // 16)


@pytest.mark.parametrize("rows,cols,tokens,want", [
    (1, 32, 1, "OK"), (1 << 24, 32768, 16, "OK"), (10007, 1408, 5, "OK"), (0, 32, 1, "INVALID_ARG"),
    (4, 0, 1, "INVALID_ARG"), (4, 48, 1, "UNSUPPORTED"), (4, 32800, 1, "UNSUPPORTED"),
    ((1 << 24) + 1, 32, 1, "UNSUPPORTED"), (4, 32, 17, "UNSUPPORTED"), (4, 32, 0, "INVALID_ARG"),
])
def test_linear_query(B, rows, cols, tokens, want):
    want = B.MOE_OK if want == "OK" else getattr(B, "MOE_ERR_" + want)
    assert status(B, B.moe_fp4_linear_workspace_query, rows, cols, tokens) == want


def test_create_refusals(B):
    dims = (256, 128, 4, 2)
    n = B.moe_fp4_workspace_query(*dims, 0, 4)
    for i, bad in [(i, 0) for i in range(6)] + [(0, A + 8), (1, A + 8), (2, A + 2), (3, A + 8), (4, A + 8), (5, A + 2)]:
        w = [A] * 6
        w[i] = bad
        assert status(B, B.moe_fp4_create, *dims, 0, 4, *w, A, n, 0) == B.MOE_ERR_INVALID_ARG
    assert status(B, B.moe_fp4_create, *dims, 0, 4, *[A] * 6, 0, n, 0) == B.MOE_ERR_INVALID_ARG
    assert status(B, B.moe_fp4_create, *dims, 0, 4, *[A] * 6, A + 8, n, 0) == B.MOE_ERR_INVALID_ARG
    assert status(B, B.moe_fp4_create, *dims, 0, 4, *[A] * 6, A, n - 1, 0) == B.MOE_ERR_WORKSPACE
    n = B.moe_fp4_linear_workspace_query(64, 64, 4)
    for i, bad in ((0, 0), (1, 0), (2, 0), (0, A + 8), (1, A + 8), (2, A + 2)):
        w = [A] * 3
        w[i] = bad
        assert status(B, B.moe_fp4_linear_create, 64, 64, 4, *w, A, n, 0) == B.MOE_ERR_INVALID_ARG
    assert status(B, B.moe_fp4_linear_create, 64, 64, 4, *[A] * 3, A, n - 1, 0) == B.MOE_ERR_WORKSPACE


def test_null_handles(B):
    L = B.lib()
    word = ctypes.c_uint32()
    assert L.moe_fp4_forward(None, A, A, A, 1, A, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_fp4_linear(None, A, 64, 1, A, 0, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_fp4_read_status(None, ctypes.byref(word), None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_forward_quantized(None, A, A, A, A, 1, None) == B.MOE_ERR_INVALID_ARG
    L.moe_fp4_destroy(None)
    out = ctypes.c_void_p(1)
    assert L.moe_fp4_create(None, 4, A, A, A, A, A, A, A, 1, None, ctypes.byref(out)) == B.MOE_ERR_INVALID_ARG
    assert not out.value
