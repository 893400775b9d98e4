"""The few-token operators launch on the current device and refuse tensors and streams of
another one (host only: tensors that say where they are, and the library's calls
replaced; none may be reached with operands of two devices)."""
import pytest
import torch

from tests.fake_device import Stream, on_device

U8, I32, F32 = torch.uint8, torch.int32, torch.float32
T, H, I, E, K = 3, 256, 128, 8, 2


@pytest.fixture
def S(monkeypatch):
    import serving_route_gb300 as S
    from serving_route_gb300 import decode
    S.calls = []
    for n in ("moe_add_rms_norm", "moe_topk_route", "moe_fp4_linear", "moe_fp4_forward"):
        monkeypatch.setattr(S.binding, n, lambda *a: S.calls.append(a))
    for n in ("moe_fp4_linear_create", "moe_fp4_create"):
        monkeypatch.setattr(S.binding, n, lambda *a: S.calls.append(a))  # (a handle of None: nothing to destroy)
    monkeypatch.setattr(S.binding, "moe_fp4_linear_workspace_query", lambda *a: 64)
    monkeypatch.setattr(S.binding, "moe_fp4_workspace_query", lambda *a: 64)
    monkeypatch.setattr(decode, "_current_device", lambda: 0, raising=False)
    yield S
    del S.calls


def norm(S, t, stream):
    S.add_rms_norm(t["x"], t["weight"], residual=t["residual"], fmt="deepseek", stream=stream,
                   out=(t["y"], t["r"], t["q"], t["s"]))


def route(S, t, stream):
    S.topk_route(t["logits"], K, scoring="sigmoid", bias=t["bias"], out=(t["idx"], t["w"]), stream=stream)


def linear_create(S, t, stream):
    S.Fp4Linear(t["codes"], t["scales"], t["glob"], stream=stream)


def linear(S, t, stream):
    lin = S.Fp4Linear.__new__(S.Fp4Linear)
    lin.rows, lin.cols = 64, H
    lin.forward(t["x"], out=t["out"], stream=stream)


def layer_bind(S, t, stream):
    S.Fp4MoELayer(H, I, E, K).bind_weights(*(t[n] for n in ("w1", "s1", "g1", "w2", "s2", "g2")), stream=stream)


def layer(S, t, stream):
    m = S.Fp4MoELayer(H, I, E, K)
    m.handle = 1
    try:
        m.forward(t["x"], t["idx"], t["w"], out=t["y"], stream=stream)
    finally:
        m.handle = None


BF = torch.bfloat16
CALLS = {
    norm: dict(x=(T, H, BF), weight=(H, BF), residual=(T, H, BF), y=(T, H, BF), r=(T, H, BF), q=(T, H, U8),
               s=(T, H // 128, U8)),
    route: dict(logits=(T, E, F32), bias=(E, F32), idx=(T, K, I32), w=(T, K, F32)),
    linear_create: dict(codes=(64, H // 2, U8), scales=(64, H // 16, U8), glob=(1, F32)),
    linear: dict(x=(T, H, BF), out=(T, 64, BF)),
    layer_bind: dict(w1=(E, 2 * I, H // 2, U8), s1=(E, 2 * I, H // 16, U8), g1=(E, F32), w2=(E, H, I // 2, U8),
                     s2=(E, H, I // 16, U8), g2=(E, F32)),
    layer: dict(x=(T, H, BF), idx=(T, K, I32), w=(T, K, F32), y=(T, H, BF)),
}


def tensors(call, dev=lambda name: 0):
    return {n: on_device(*s[:-1], dtype=s[-1], dev=dev(n)) for n, s in CALLS[call].items()}


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_taken_on_the_current_device(S, call):
    call(S, tensors(call), Stream())
    assert len(S.calls) == 1


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS.items() for n in names],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
@pytest.mark.parametrize("dev", [1, -1])
def test_one_tensor_elsewhere(S, call, name, dev):
    with pytest.raises(AssertionError):
        call(S, tensors(call, lambda n: dev if n == name else 0), Stream())
    assert not S.calls


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_all_on_another_device(S, call):
    with pytest.raises(AssertionError):
        call(S, tensors(call, lambda n: 1), Stream(1))
    with pytest.raises(AssertionError):
        call(S, tensors(call), Stream(1))
    assert not S.calls
