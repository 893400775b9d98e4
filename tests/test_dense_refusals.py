"""Host-side checks of the dense products (no GPU needed): what the calls refuse they refuse
before any CUDA call, the workspace queries apply the documented rules, and tensors and
streams of another device than the current one do not reach the library.  The addresses
below are numbers, not memory: no call here reads them."""
import ctypes

import pytest
import torch

from tests.fake_device import Stream, on_device

A = 0x7000000000  # a 16-byte aligned "device address"
BF, HF, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


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


@pytest.mark.parametrize("rows,cols,tokens,want", [
    (1, 128, 1, "OK"), (10007, 1408, 8192, "OK"), (1 << 24, 128, 1, "OK"), (128, 32768, 1 << 24, "OK"),
    (0, 128, 1, "ERR_INVALID_ARG"), (1, 0, 1, "ERR_INVALID_ARG"), (1, 128, 0, "ERR_INVALID_ARG"),
    (1, 64, 1, "ERR_UNSUPPORTED"), (1, 200, 1, "ERR_UNSUPPORTED"), (1, 32896, 1, "ERR_UNSUPPORTED"),
    ((1 << 24) + 1, 128, 1, "ERR_UNSUPPORTED"), (1, 128, (1 << 24) + 1, "ERR_UNSUPPORTED")])
def test_linear_query(B, rows, cols, tokens, want):
    assert status(B, B.moe_fp8_linear_workspace_query, rows, cols, tokens) == getattr(B, "MOE_" + want)
    if want == "OK":
        n = B.moe_fp8_linear_workspace_query(rows, cols, tokens)
        assert n >= tokens * (cols + cols // 128) + (rows + 127) // 128 * (cols // 128)


@pytest.mark.parametrize("hidden,inter,tokens,want", [
    (8, 8, 1, "OK"), (7168, 2048, 8192, "OK"), (65536, 65536, 1, "OK"),
    (0, 8, 1, "ERR_INVALID_ARG"), (8, 0, 1, "ERR_INVALID_ARG"), (8, 8, 0, "ERR_INVALID_ARG"),
    (12, 8, 1, "ERR_UNSUPPORTED"), (8, 4, 1, "ERR_UNSUPPORTED"), (65544, 8, 1, "ERR_UNSUPPORTED"),
    (8, 65544, 1, "ERR_UNSUPPORTED"), (8, 8, (1 << 24) + 1, "ERR_UNSUPPORTED")])
def test_mlp_query(B, hidden, inter, tokens, want):
    assert status(B, B.moe_mlp_workspace_query, hidden, inter, tokens) == getattr(B, "MOE_" + want)
    if want == "OK":
        assert B.moe_mlp_workspace_query(hidden, inter, tokens) >= 6 * tokens * inter


@pytest.mark.parametrize("change,want", [
    (dict(codes=0), "INVALID_ARG"), (dict(codes=A + 8), "INVALID_ARG"), (dict(scales=0), "INVALID_ARG"),
    (dict(scales=A + 2), "INVALID_ARG"), (dict(ws=0), "INVALID_ARG"), (dict(ws=A + 4), "INVALID_ARG"),
    (dict(n=1024), "WORKSPACE"), (dict(flags=1), "UNSUPPORTED"), (dict(cols=100), "UNSUPPORTED"), (dict(tokens=0), "INVALID_ARG")])
def test_linear_create(B, change, want):
    kw = {**dict(rows=64, cols=256, flags=0, tokens=4, codes=A, scales=A, ws=A, n=1 << 20, stream=0), **change}
    assert status(B, B.moe_fp8_linear_create, *kw.values()) == getattr(B, "MOE_ERR_" + want)


@pytest.mark.parametrize("change,want", [
    (dict(w1=0), "INVALID_ARG"), (dict(w2=0), "INVALID_ARG"), (dict(w1=A + 8), "INVALID_ARG"), (dict(w2=A + 2), "INVALID_ARG"),
    (dict(ws=0), "INVALID_ARG"), (dict(ws=A + 8), "INVALID_ARG"), (dict(n=2048), "WORKSPACE"), (dict(act=2), "UNSUPPORTED"),
    (dict(act=-1), "UNSUPPORTED"), (dict(flags=0x21), "UNSUPPORTED"), (dict(hidden=20), "UNSUPPORTED")])
def test_mlp_create(B, change, want):
    kw = {**dict(hidden=64, inter=32, fp16=0, act=0, flags=0, tokens=4, w1=A, w2=A, ws=A, n=1 << 20, stream=0), **change}
    assert status(B, B.moe_mlp_create, *kw.values()) == getattr(B, "MOE_ERR_" + want)


def test_handles_of_nothing(B):
    """NULL handles are refused, and destroying one is a no-op."""
    L = B.lib()
    bits = ctypes.c_uint32()
    for f, args in ((L.moe_fp8_linear, (A, 256, 1, A, 0, 0)), (L.moe_fp8_linear_quantized, (A, A, 1, A, 0, 0)),
                    (L.moe_mlp_forward, (A, 64, 1, A, None, 0, 0)),
                    (L.moe_mlp_backward, (A, 64, A, 64, A, 0, 1, A, A, A, 0, 0, 0)),
                    (L.moe_fp8_linear_read_status, (ctypes.byref(bits), 0)), (L.moe_mlp_read_status, (ctypes.byref(bits), 0))):
        assert f(None, *args) == B.MOE_ERR_INVALID_ARG
    assert L.moe_fp8_linear_create(64, 256, 0, 4, A, A, A, 1 << 20, None, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_mlp_create(64, 32, 0, 0, 0, 4, A, A, A, 1 << 20, None, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_fp8_linear_workspace_query(64, 256, 4, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_mlp_workspace_query(64, 32, 4, None) == B.MOE_ERR_INVALID_ARG
    L.moe_fp8_linear_destroy(None)
    L.moe_mlp_destroy(None)


# ---------------------------------------------------------------------------- the Python classes
T, H, I, ROWS = 3, 256, 128, 200


@pytest.fixture
def S(monkeypatch):
    import serving_route_gb300 as S
    from serving_route_gb300 import dense
    S.calls = []
    for n in ("moe_fp8_linear_create", "moe_mlp_create", "moe_fp8_linear", "moe_fp8_linear_quantized", "moe_mlp_forward",
              "moe_mlp_backward"):
        monkeypatch.setattr(S.binding, n, lambda *a: S.calls.append(a))  # (handles of None: nothing to destroy)
    for n in ("moe_fp8_linear_workspace_query", "moe_mlp_workspace_query"):
        monkeypatch.setattr(S.binding, n, lambda *a: 64)
    monkeypatch.setattr(dense, "_current_device", lambda: 0)
    monkeypatch.setattr(dense, "_current_stream", lambda dev: 0)
    yield S
    del S.calls


def tensors():
    return dict(codes=on_device(ROWS, H, dtype=U8), scales=on_device(2, 2, dtype=F32), x=on_device(T, H),
                xq=on_device(T, H, dtype=U8), xs=on_device(T, 2, dtype=U8), out=on_device(T, ROWS),
                w1=on_device(2 * I, H), w2=on_device(H, I), y=on_device(T, H), saved=on_device(T, 2 * I, dtype=F32),
                dy=on_device(T, H), dx=on_device(T, H), dw1=on_device(2 * I, H), dw2=on_device(H, I))


def made(cls, **kw):
    o = cls.__new__(cls)
    o.__dict__.update(kw)
    return o


CALLS = {
    "linear_create": (("codes", "scales"), lambda S, t, s: S.Fp8Linear(t["codes"], t["scales"], max_tokens=T, stream=s)),
    "linear": (("x", "out"), lambda S, t, s: made(S.Fp8Linear, rows=ROWS, cols=H).forward(t["x"], out=t["out"], stream=s)),
    "linear_quantized": (("xq", "xs", "out"), lambda S, t, s: made(S.Fp8Linear, rows=ROWS, cols=H).forward_quantized(
        t["xq"], t["xs"], out=t["out"], stream=s)),
    "mlp_create": (("w1", "w2"), lambda S, t, s: S.GatedMlp(t["w1"], t["w2"], max_tokens=T, stream=s)),
    "mlp": (("x", "y", "saved"), lambda S, t, s: made(S.GatedMlp, H=H, I=I, dtype=BF).forward(
        t["x"], out=t["y"], saved=t["saved"], stream=s)),
    "mlp_backward": (("dy", "x", "saved", "dx", "dw1", "dw2"), lambda S, t, s: made(S.GatedMlp, H=H, I=I, dtype=BF).backward(
        t["dy"], t["x"], t["saved"], out=(t["dx"], t["dw1"], t["dw2"]), stream=s)),
}


@pytest.mark.parametrize("call", CALLS)
def test_operands_of_one_device(S, call):
    names, run = CALLS[call]
    run(S, tensors(), Stream())
    run(S, tensors(), None)
    assert len(S.calls) == 2
    for n in names:  # each operand elsewhere, and on the host
        for dev in (1, -1):
            t = tensors()
            t[n].dev = dev
            with pytest.raises(AssertionError):
                run(S, t, Stream())
    t = tensors()
    for n in names:
        t[n].dev = 1
    with pytest.raises(AssertionError):
        run(S, t, Stream(1))
    with pytest.raises(AssertionError):
        run(S, tensors(), Stream(1))
    assert len(S.calls) == 2


@pytest.mark.parametrize("call,name,bad", [
    ("linear_create", "codes", on_device(ROWS, H)), ("linear_create", "scales", on_device(1, 2, dtype=F32)),
    ("linear_create", "scales", on_device(2, 2)), ("linear", "x", on_device(T, H, dtype=HF)),
    ("linear", "x", on_device(T, H // 2)), ("linear", "x", on_device(H, T).t()), ("linear", "out", on_device(T + 1, ROWS)),
    ("linear", "out", on_device(T, ROWS, dtype=HF)), ("linear", "out", on_device(ROWS, T).t()),
    ("linear_quantized", "xq", on_device(T, 2 * H, dtype=U8)[:, :H]), ("linear_quantized", "xs", on_device(T, 3, dtype=U8)),
    ("linear_quantized", "xs", on_device(T, 2)), ("mlp_create", "w1", on_device(2 * I, H, dtype=HF)),
    ("mlp_create", "w1", on_device(I, H)), ("mlp_create", "w2", on_device(I, H).t()), ("mlp_create", "w2", on_device(H, I, dtype=F32)),
    ("mlp", "x", on_device(T, H, dtype=HF)), ("mlp", "y", on_device(T, H, dtype=F32)), ("mlp", "saved", on_device(T, 2 * I, dtype=HF)),
    ("mlp", "saved", on_device(T, I, dtype=F32)), ("mlp_backward", "dy", on_device(T + 1, H)),
    ("mlp_backward", "dx", on_device(T, H, dtype=F32)), ("mlp_backward", "dw1", on_device(2 * I, H, dtype=F32)),
    ("mlp_backward", "dw2", on_device(H, I, dtype=HF)), ("mlp_backward", "saved", on_device(T, 2 * I, dtype=HF))])
def test_wrong_operands(S, call, name, bad):
    t = tensors()
    t[name] = bad
    with pytest.raises(AssertionError):
        CALLS[call][1](S, t, Stream())
    assert not S.calls


def test_accumulation_needs_float_gradients(S):
    t, mlp = tensors(), made(S.GatedMlp, H=H, I=I, dtype=BF)
    with pytest.raises(AssertionError):
        mlp.backward(t["dy"], t["x"], t["saved"], out=(t["dx"], t["dw1"], t["dw2"]), accumulate=True, stream=Stream())
    f = on_device(2 * I, H, dtype=F32), on_device(H, I, dtype=F32)
    mlp.backward(t["dy"], t["x"], t["saved"], out=(t["dx"], *f), accumulate=True, stream=Stream())
    assert len(S.calls) == 1
    with pytest.raises(AssertionError):
        S.GatedMlp(t["w1"], t["w2"], max_tokens=T, activation="relu")
