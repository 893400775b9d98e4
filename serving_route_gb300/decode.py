"""The operators around the MoE layer for few tokens: the residual norm with its
8-bit output, the choice of experts, products of a few vectors with an NVFP4
matrix, and the whole layer on NVFP4 experts.  PyTorch provides device memory
and streams only; every computation is a kernel of the library.

Given `out` buffers the calls allocate nothing and can be captured in a CUDA
graph.  Tensors used on another stream than the one they were made on are the
caller's to order (and to keep alive), as for MegaMoELayer.  The kernels run on the
current device: all tensors (and the stream) of a call are of that device, else it is
refused.
"""
from __future__ import annotations

import torch

from . import binding as B
from .layer import _stream_ptr

_Q_FORMATS = {"deepseek": 0, "mxfp8": B.MOE_FLAG_MXFP8, "per_tensor": B.MOE_FLAG_PER_TENSOR}
_Q_BLOCK = {"deepseek": 128, "mxfp8": 32}


_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


# The current device, which the library launches on (a tensor on the host is on device
# -1), and the raw handle of its current stream, without making a Stream object of it.
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _given_stream(stream, dev: int) -> int:
    assert getattr(stream, "device_index", dev) == dev
    return stream.cuda_stream


# The checks below are written out, not shared: at a few microseconds a call
# the calls of helper functions are a good part of these operators' time for
# one token.


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                 residual: torch.Tensor | None = None, fmt: str | None = None, scale: float = 1.0,
                 out=None, stream=None):
    """r = bf16(x + residual) (r = x without one), y = r * rsqrt(mean(r^2) + eps) * weight.

    x, residual: BF16 [T, H] (rows may be strided); weight: BF16 [H].
    fmt: None, or the 8-bit format of the second output: "deepseek" (a
    power-of-two scale per 128 columns), "mxfp8" (per 32) or "per_tensor" (the
    static `scale`).  Returns (y, r, q, q_scale): y BF16 [T, H], r BF16 [T, H]
    or None, q uint8 E4M3 codes [T, H] or None, q_scale uint8 E8M0 bytes
    [T, H/128 or H/32] or None.  out: such a tuple of buffers to write
    (y may be x, r may be residual; y may be None where q is wanted)."""
    shape = x.shape
    T, H = shape
    ldx, one = x.stride()
    dev = x.get_device()
    assert x.dtype is _BF16 and dev == _current_device() and (one == 1 or H == 1)
    assert weight.dtype is _BF16 and weight.get_device() == dev and weight.shape == (H,) and weight.is_contiguous()
    if T <= 1:  # the stride of a single row says nothing
        ldx = H
    res = ldr = 0
    if residual is not None:
        ldr, one = residual.stride()
        assert residual.dtype is _BF16 and residual.get_device() == dev and residual.shape == shape
        assert one == 1 or H == 1
        res = residual.data_ptr()
        if T <= 1:
            ldr = H
    block = 0
    if fmt is not None:
        assert fmt in _Q_FORMATS
        block = _Q_BLOCK.get(fmt, 0)
        if block and H % block:  # the library's refusal, before a scale buffer of a wrong shape is made
            raise B.MoEError(B.MOE_ERR_UNSUPPORTED, "moe_add_rms_norm")
    if out is None:
        y = torch.empty(T, H, dtype=_BF16, device=x.device)
        r = torch.empty_like(y) if residual is not None else None
        q = torch.empty(T, H, dtype=_U8, device=x.device) if fmt else None
        s = torch.empty(T, H // block, dtype=_U8, device=x.device) if block else None
        out = y, r, q, s
    else:
        y, r, q, s = out
        assert y is None or (y.dtype is _BF16 and y.get_device() == dev and y.shape == shape and y.is_contiguous())
        if residual is None:
            assert r is None
        else:
            assert r.dtype is _BF16 and r.get_device() == dev and r.shape == shape and r.is_contiguous()
        if fmt is None:
            assert q is None and s is None
        else:
            assert q.dtype is _U8 and q.get_device() == dev and q.shape == shape and q.is_contiguous()
            if block:
                assert s.dtype is _U8 and s.get_device() == dev and s.shape == (T, H // block) and s.is_contiguous()
            else:
                assert s is None
    B.moe_add_rms_norm(x.data_ptr(), ldx, res, ldr, weight.data_ptr(), eps, T, H,
                       0 if r is None else r.data_ptr(), 0 if y is None else y.data_ptr(),
                       0 if q is None else q.data_ptr(), 0 if s is None else s.data_ptr(),
                       _Q_FORMATS[fmt] if fmt is not None else 0, scale,
                       _current_stream(dev) if stream is None else _given_stream(stream, dev))
    return y, r, q, s


def topk_route(logits: torch.Tensor, top_k: int, *, scoring: str = "softmax",
               bias: torch.Tensor | None = None, num_groups: int = 1, top_groups: int = 1,
               renormalize: bool = True, scale: float = 1.0, out=None, stream=None):
    """Gate logits (float32 or BF16 [T, E], rows may be strided) to expert ids
    (int32 [T, top_k], descending, ties to the lowest) and weights (float32),
    as the forwards take them.  scoring "softmax" chooses by the logit,
    "sigmoid" by sigmoid + bias (float32 [E]); weights never hold the bias.
    The choice is limited to the top_groups best of num_groups equal groups (a
    group's score: its largest logit, or the sum of its two largest biased
    scores).  Logits of -inf mask an expert; slots left over get id -1.
    A row with a NaN gets NaN weights, and at least one id."""
    T, E = logits.shape
    ld, one = logits.stride()
    bf16 = logits.dtype is _BF16
    dev = logits.get_device()
    assert (bf16 or logits.dtype is _F32) and dev == _current_device() and (one == 1 or E == 1)
    assert scoring == "softmax" or scoring == "sigmoid"
    assert bias is None or (bias.dtype is _F32 and bias.get_device() == dev and bias.shape == (E,)
                            and bias.is_contiguous())
    if out is None:
        idx = torch.empty(T, top_k, dtype=_I32, device=logits.device)
        w = torch.empty(T, top_k, dtype=_F32, device=logits.device)
    else:
        idx, w = out
        shape = (T, top_k)
        assert idx.dtype is _I32 and idx.get_device() == dev and idx.shape == shape and idx.is_contiguous()
        assert w.dtype is _F32 and w.get_device() == dev and w.shape == shape and w.is_contiguous()
    B.moe_topk_route(logits.data_ptr(), bf16, E if T <= 1 else ld, 0 if bias is None else bias.data_ptr(), T, E,
                     top_k, scoring == "sigmoid", num_groups, top_groups, renormalize, scale, idx.data_ptr(),
                     w.data_ptr(), _current_stream(dev) if stream is None else _given_stream(stream, dev))
    return idx, w


def _dense(t: torch.Tensor, dtype, shape, dev: int) -> bool:
    return t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()


class _Fp4Handle:
    handle = None

    def read_status(self, stream=None):
        """(status code, device status bits) of the latest forward; synchronises the stream."""
        return B.moe_fp4_read_status(self.handle, _stream_ptr(stream))

    def close(self) -> None:
        if self.handle:
            B.moe_fp4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Fp4Linear(_Fp4Handle):
    """y = x W^T for 1..max_tokens (<= 16) BF16 vectors and one NVFP4 matrix.

    codes uint8 [rows, cols/2] (even column in the low nibble), block_scales
    uint8 [rows, cols/16] (E4M3), global_scale float32 [1], all on the GPU; the
    object keeps them and its own workspace.  cols is a multiple of 32.
    Forwards of one object must not overlap on the GPU."""

    def __init__(self, codes: torch.Tensor, block_scales: torch.Tensor, global_scale: torch.Tensor, *,
                 max_tokens: int = 16, stream=None):
        rows, cols = codes.shape[0], 2 * codes.shape[1]
        n = B.moe_fp4_linear_workspace_query(rows, cols, max_tokens)
        dev = codes.get_device()
        assert dev == _current_device()
        assert _dense(codes, torch.uint8, (rows, cols // 2), dev)
        assert _dense(block_scales, torch.uint8, (rows, cols // 16), dev)
        assert _dense(global_scale, torch.float32, (1,), dev)
        self.rows, self.cols, self.max_tokens = rows, cols, max_tokens
        self.weights = (codes, block_scales, global_scale)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=codes.device)
        self.handle = B.moe_fp4_linear_create(rows, cols, max_tokens, codes.data_ptr(),
                                              block_scales.data_ptr(), global_scale.data_ptr(),
                                              self.workspace.data_ptr(), n,
                                              _current_stream(dev) if stream is None else _given_stream(stream, dev))

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, *,
                out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """x BF16 [T, cols] (rows may be strided by a multiple of 8) -> [T, rows] in
        out_dtype (bfloat16 or float32) or in `out`'s type; `out` may not overlap x."""
        T, cols = x.shape
        ldx, one = x.stride()
        dev = x.get_device()
        assert x.dtype is _BF16 and dev == _current_device() and cols == self.cols and one == 1
        if out is None:
            assert out_dtype is _BF16 or out_dtype is _F32
            out = torch.empty(T, self.rows, dtype=out_dtype, device=x.device)
        f32 = out.dtype is _F32
        assert (f32 or out.dtype is _BF16) and out.get_device() == dev and out.shape == (T, self.rows)
        assert out.is_contiguous()
        B.moe_fp4_linear(self.handle, x.data_ptr(), cols if T <= 1 else ldx, T, out.data_ptr(), f32,
                         _current_stream(dev) if stream is None else _given_stream(stream, dev))
        return out


class Fp4MoELayer(_Fp4Handle):
    """The whole MoE layer for 1..max_tokens (<= 16) tokens on NVFP4 experts, read
    in the checkpoint's layout; same inputs and routes as MegaMoELayer.forward.
    The object keeps the bound weights and its own workspace.  Forwards of one
    object must not overlap on the GPU."""

    def __init__(self, hidden: int, inter: int, num_experts: int, top_k: int, *, max_tokens: int = 16,
                 check_routes: bool = True, watchdog_test: bool = False):
        self.H, self.I, self.E, self.K = hidden, inter, num_experts, top_k
        self.max_tokens = max_tokens
        self.flags = ((B.MOE_FLAG_CHECK_ROUTES if check_routes else 0)
                      | (B.MOE_FLAG_WATCHDOG_TEST if watchdog_test else 0))
        self._ws_bytes = B.moe_fp4_workspace_query(hidden, inter, num_experts, top_k, self.flags, max_tokens)

    def bind_weights(self, w1, w1_scales, w1_global, w2, w2_scales, w2_global, stream=None) -> None:
        """w1 uint8 [E, 2I, H/2] (gate rows, then up rows) with scales uint8 [E, 2I, H/16]
        and float32 [E]; w2 uint8 [E, H, I/2] likewise."""
        E, H, I = self.E, self.H, self.I
        dev = w1.get_device()
        assert dev == _current_device()
        assert _dense(w1, torch.uint8, (E, 2 * I, H // 2), dev) and _dense(w2, torch.uint8, (E, H, I // 2), dev)
        assert _dense(w1_scales, torch.uint8, (E, 2 * I, H // 16), dev)
        assert _dense(w2_scales, torch.uint8, (E, H, I // 16), dev)
        assert _dense(w1_global, torch.float32, (E,), dev) and _dense(w2_global, torch.float32, (E,), dev)
        self.close()
        self.weights = (w1, w1_scales, w1_global, w2, w2_scales, w2_global)
        self.workspace = torch.empty(self._ws_bytes, dtype=torch.uint8, device=w1.device)
        self.handle = B.moe_fp4_create(H, I, E, self.K, self.flags, self.max_tokens,
                                       *(t.data_ptr() for t in self.weights), self.workspace.data_ptr(),
                                       self._ws_bytes,
                                       _current_stream(dev) if stream is None else _given_stream(stream, dev))

    def forward(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x BF16 [T, H], topk_idx int32 [T, K] (-1: masked slot), topk_w float32 [T, K] -> BF16 [T, H].
        `out` may be x."""
        if self.handle is None:
            raise B.MoEError(B.MOE_ERR_NOT_BOUND, "moe_fp4_forward")
        shape, routes = x.shape, topk_idx.shape
        T, H = shape
        dev = x.get_device()
        assert x.dtype is _BF16 and dev == _current_device() and H == self.H and x.is_contiguous()
        assert topk_idx.dtype is _I32 and topk_idx.get_device() == dev and routes == (T, self.K)
        assert topk_w.dtype is _F32 and topk_w.get_device() == dev and topk_w.shape == routes
        assert topk_idx.is_contiguous() and topk_w.is_contiguous()
        if out is None:
            out = torch.empty(T, H, dtype=_BF16, device=x.device)
        else:
            assert out.dtype is _BF16 and out.get_device() == dev and out.shape == shape and out.is_contiguous()
        B.moe_fp4_forward(self.handle, x.data_ptr(), topk_idx.data_ptr(), topk_w.data_ptr(), T,
                          out.data_ptr(), _current_stream(dev) if stream is None else _given_stream(stream, dev))
        return out
