"""The dense products beside the MoE layer, for any number of tokens: a linear in the
layer's FP8 format and a gated feed-forward block (a shared expert, a dense layer) with its
gradients.  PyTorch provides device memory and streams only; every computation is a
kernel of the library.

Given their buffers the calls allocate nothing and can be captured in a CUDA graph.
Tensors used on another stream than the one they were made on are the caller's to order
(and to keep alive), as for MegaMoELayer.  The kernels run on the current device: all
tensors (and the stream) of a call are of that device, else it is refused.  Calls of one
object must not overlap on the GPU: they share its workspace.
"""
from __future__ import annotations

import torch

from . import binding as B
from .decode import _BF16, _F32, _U8, _current_device, _current_stream, _dense, _given_stream
from .layer import _stream_ptr

_F16 = torch.float16
_ACTS = {"silu": B.MOE_ACT_SILU, "gelu": B.MOE_ACT_GELU_TANH}


class _Handle:
    handle = None

    def close(self) -> None:
        if self.handle:
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _launch(p) -> dict:
    return {n: getattr(p, n) for n in ("pairs", "width", "split", "tiles")}


def _rows(t: torch.Tensor, dtype, cols: int, dev: int) -> bool:
    """Whether t is [T, cols] of dtype, its rows contiguous (they may be strided)."""
    return (t.dtype is dtype and t.get_device() == dev and t.dim() == 2 and t.shape[1] == cols
            and t.stride(1) == 1)


class Fp8Linear(_Handle):
    """y = x W^T for up to max_tokens rows and one FP8 matrix in MegaMoELayer's default format.

    codes uint8 E4M3 [rows, cols], scales float32 [ceil(rows/128), cols/128] (powers of
    two, one per 128x128 block: MegaMoELayer.quantize_weights of [1, rows, cols]), on the
    GPU.  cols is a multiple of 128; rows need not be.  The object keeps the codes and
    its own workspace."""

    _destroy = staticmethod(B.moe_fp8_linear_destroy)

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, *, max_tokens: int, watchdog_test: bool = False,
                 stream=None):
        rows, cols = codes.shape
        n = B.moe_fp8_linear_workspace_query(rows, cols, max_tokens)
        dev = codes.get_device()
        assert dev == _current_device()
        assert _dense(codes, _U8, (rows, cols), dev)
        assert _dense(scales, _F32, ((rows + 127) // 128, cols // 128), dev)
        self.rows, self.cols, self.max_tokens = rows, cols, max_tokens
        self.codes = codes
        self.workspace = torch.empty(n, dtype=_U8, device=codes.device)
        self.handle = B.moe_fp8_linear_create(rows, cols, B.MOE_FLAG_WATCHDOG_TEST if watchdog_test else 0,
                                              max_tokens, codes.data_ptr(), scales.data_ptr(),
                                              self.workspace.data_ptr(), n,
                                              _current_stream(dev) if stream is None else _given_stream(stream, dev))

    def _out(self, T: int, out, out_dtype, device, dev: int):
        if out is None:
            assert out_dtype is _BF16 or out_dtype is _F32
            return torch.empty(T, self.rows, dtype=out_dtype, device=device)
        assert (out.dtype is _F32 or out.dtype is _BF16) and out.get_device() == dev
        assert out.shape == (T, self.rows) and out.is_contiguous()
        return out

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, *,
                out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """x BF16 [T, cols] (rows may be strided by a multiple of 8), rounded to E4M3 with a
        power-of-two scale per 128 columns -> [T, rows] in out_dtype (bfloat16 or float32) or in
        `out`'s type; `out` may not overlap x.  A row with a NaN or an infinity gives NaN."""
        T = x.shape[0]
        dev = x.get_device()
        assert dev == _current_device() and _rows(x, _BF16, self.cols, dev)
        out = self._out(T, out, out_dtype, x.device, dev)
        B.moe_fp8_linear(self.handle, x.data_ptr(), self.cols if T <= 1 else x.stride(0), T, out.data_ptr(),
                         out.dtype is _F32, _current_stream(dev) if stream is None else _given_stream(stream, dev))
        return out

    def forward_quantized(self, xq: torch.Tensor, xq_scale: torch.Tensor, out: torch.Tensor | None = None, *,
                          out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """forward() of rows in that form already, as add_rms_norm(fmt="deepseek") gives them: xq
        uint8 E4M3 codes [T, cols], xq_scale uint8 E8M0 bytes [T, cols/128]."""
        T = xq.shape[0]
        dev = xq.get_device()
        assert dev == _current_device() and _dense(xq, _U8, (T, self.cols), dev)
        assert _dense(xq_scale, _U8, (T, self.cols // 128), dev)
        out = self._out(T, out, out_dtype, xq.device, dev)
        B.moe_fp8_linear_quantized(self.handle, xq.data_ptr(), xq_scale.data_ptr(), T, out.data_ptr(),
                                   out.dtype is _F32,
                                   _current_stream(dev) if stream is None else _given_stream(stream, dev))
        return out

    def plan(self, num_tokens: int, quantized: bool = False) -> dict:
        """How forward (or forward_quantized) divides num_tokens tokens: pairs, width, split, tiles."""
        return _launch(B.moe_fp8_linear_plan(self.handle, num_tokens, quantized))

    def read_status(self, stream=None):
        """(status code, device status bits) since the last read; synchronises the stream."""
        return B.moe_fp8_linear_read_status(self.handle, _stream_ptr(stream))


class GatedMlp(_Handle):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T for up to max_tokens rows, in BF16 or FP16, and its gradients
    (by backward(): the calls take no part in autograd).

    w1 [2I, H] (gate rows, then up rows), w2 [H, I], of one type, on the GPU; H and I
    multiples of 8.  activation: "silu", or "gelu" in its tanh form.  The object keeps
    the weights, which every call reads where they are (an optimiser may change them in
    place), and its own workspace of 6 max_tokens I bytes (2 of them are the forward's)."""

    _destroy = staticmethod(B.moe_mlp_destroy)

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, *, max_tokens: int, activation: str = "silu",
                 watchdog_test: bool = False, watchdog_last_test: bool = False, stream=None):
        H, I = w2.shape
        assert activation in _ACTS
        n = B.moe_mlp_workspace_query(H, I, max_tokens)
        dev, dtype = w1.get_device(), w1.dtype
        assert dev == _current_device() and (dtype is _BF16 or dtype is _F16)
        assert _dense(w1, dtype, (2 * I, H), dev) and _dense(w2, dtype, (H, I), dev)
        self.H, self.I, self.max_tokens, self.dtype = H, I, max_tokens, dtype
        self.weights = (w1, w2)
        self.workspace = torch.empty(n, dtype=_U8, device=w1.device)
        self.handle = B.moe_mlp_create(H, I, dtype is _F16, _ACTS[activation],
                                       (B.MOE_FLAG_WATCHDOG_TEST if watchdog_test else 0)
                                       | (B.MOE_FLAG_WATCHDOG_LAST_TEST if watchdog_last_test else 0),
                                       max_tokens, w1.data_ptr(), w2.data_ptr(), self.workspace.data_ptr(), n,
                                       _current_stream(dev) if stream is None else _given_stream(stream, dev))

    def _saved(self, saved: torch.Tensor, T: int, dev: int) -> bool:
        return _dense(saved, _F32 if saved.dtype is _F32 else self.dtype, (T, 2 * self.I), dev)

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, *, saved: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """x [T, H] in the weights' type (rows may be strided by a multiple of 8) -> [T, H].
        `out` may be x.  saved: a buffer [T, 2I], float32 or in the weights' type, that
        takes gate and up before the activation for backward() (in FP16 what is beyond 65504 is
        infinite, and its gradients infinite or NaN)."""
        T = x.shape[0]
        dev = x.get_device()
        assert dev == _current_device() and _rows(x, self.dtype, self.H, dev)
        if out is None:
            out = torch.empty(T, self.H, dtype=self.dtype, device=x.device)
        assert _dense(out, self.dtype, (T, self.H), dev)
        assert saved is None or self._saved(saved, T, dev)
        B.moe_mlp_forward(self.handle, x.data_ptr(), self.H if T <= 1 else x.stride(0), T, out.data_ptr(),
                          0 if saved is None else saved.data_ptr(), saved is not None and saved.dtype is _F32,
                          _current_stream(dev) if stream is None else _given_stream(stream, dev))
        return out

    def backward(self, dy: torch.Tensor, x: torch.Tensor, saved: torch.Tensor, out=None, *,
                 accumulate: bool = False, stream=None):
        """(dx, dw1, dw2) from dy [T, H], the forward's x and what it saved (rows of dy
        and x may be strided by a multiple of 8).  out: such a tuple of buffers; one that is None
        is not computed.  dx is in the weights' type, dw1 [2I, H] and dw2 [H, I] in it
        or both float32 (float32 given as `out`, and then with accumulate added to what they hold)."""
        T, H, I = x.shape[0], self.H, self.I
        dev = x.get_device()
        assert dev == _current_device() and _rows(x, self.dtype, H, dev)
        assert _rows(dy, self.dtype, H, dev) and dy.shape[0] == T and self._saved(saved, T, dev)
        if out is None:
            out = (torch.empty(T, H, dtype=self.dtype, device=x.device),
                   torch.empty(2 * I, H, dtype=self.dtype, device=x.device),
                   torch.empty(H, I, dtype=self.dtype, device=x.device))
        dx, dw1, dw2 = out
        grad = next((t.dtype for t in (dw1, dw2) if t is not None), self.dtype)
        assert grad is self.dtype or grad is _F32
        assert grad is _F32 or not accumulate
        assert dx is None or _dense(dx, self.dtype, (T, H), dev)
        assert dw1 is None or _dense(dw1, grad, (2 * I, H), dev)
        assert dw2 is None or _dense(dw2, grad, (H, I), dev)
        B.moe_mlp_backward(self.handle, dy.data_ptr(), H if T <= 1 else dy.stride(0), x.data_ptr(),
                           H if T <= 1 else x.stride(0), saved.data_ptr(), saved.dtype is _F32, T,
                           *(0 if t is None else t.data_ptr() for t in out), grad is _F32, accumulate,
                           _current_stream(dev) if stream is None else _given_stream(stream, dev))
        return dx, dw1, dw2

    def plan(self, num_tokens: int) -> dict:
        """The launches of forward ("gate", "down") and backward ("dh", "gradients") on num_tokens
        tokens: pairs, width, split, tiles of each."""
        return dict(zip(("gate", "down", "dh", "gradients"), map(_launch, B.moe_mlp_plan(self.handle, num_tokens))))

    def read_status(self, stream=None):
        """(status code, device status bits) since the last read; synchronises the stream."""
        return B.moe_mlp_read_status(self.handle, _stream_ptr(stream))
