"""MegaMoELayer.forward_quantized refuses routes that the kernels would read past
(host only: the library's call is replaced, and must not be reached)."""
import pytest
import torch

from tests.fake_device import Stream, on_device

T, H, E, K = 5, 256, 8, 2


@pytest.fixture
def layer(monkeypatch):
    import serving_route_gb300 as S
    m = S.MegaMoELayer.__new__(S.MegaMoELayer)
    m.H, m.E, m.K, m.fmt, m.handle, m.out = H, E, K, "deepseek", 1, torch.zeros(T, H)
    m.calls = []
    monkeypatch.setattr(S.binding, "moe_forward_quantized", lambda *a: m.calls.append(a))
    yield m
    m.handle = None  # there is nothing to destroy


def args(**change):
    a = dict(xq=on_device(T, H, dtype=torch.uint8), xq_scale=on_device(T, H // 128, dtype=torch.uint8),
             topk_idx=on_device(T, K, dtype=torch.int32), topk_w=on_device(T, K, dtype=torch.float32),
             stream=Stream())
    return {**a, **change}


@pytest.mark.parametrize("rows", [T, T + 3])
def test_taken(layer, rows):
    layer.forward_quantized(**args(topk_idx=on_device(rows, K, dtype=torch.int32),
                                   topk_w=on_device(rows, K, dtype=torch.float32)))
    assert len(layer.calls) == 1


@pytest.mark.parametrize("bad", [
    lambda dt: on_device(T - 1, K, dtype=dt), lambda dt: on_device(T, K - 1, dtype=dt),
    lambda dt: on_device(T, K + 1, dtype=dt), lambda dt: on_device(T * K, dtype=dt),
    lambda dt: on_device(K, T, dtype=dt).t(), lambda dt: on_device(2 * T, K, dtype=dt)[::2],
    lambda dt: torch.zeros(T, K, dtype=dt)])
def test_refused(layer, bad):
    for change in (dict(topk_idx=bad(torch.int32)), dict(topk_w=bad(torch.float32))):
        with pytest.raises(AssertionError):
            layer.forward_quantized(**args(**change))
    assert not layer.calls
