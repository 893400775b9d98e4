"""The operators around the MoE layer for few tokens: the residual norm with its
8-bit output, the choice of experts, products of a few vectors with an NVFP4
matrix, and the whole layer on NVFP4 experts.  PyTorch provides device memory
and streams only; every computation is a kernel of the library.

Given `out` buffers the calls allocate nothing and can be captured in a CUDA
graph.  Tensors used on another stream than the one they were made on are the
caller's to order (and to keep alive), as for MegaMoELayer.
"""
from __future__ import annotations

import torch

from . import binding as B
from .layer import _stream_ptr

_Q_FORMATS = {"deepseek": 0, "mxfp8": B.MOE_FLAG_MXFP8, "per_tensor": B.MOE_FLAG_PER_TENSOR}
_Q_BLOCK = {"deepseek": 128, "mxfp8": 32}


def _dense(t: torch.Tensor, dtype, shape) -> bool:
    return t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()


def _rows_ok(t: torch.Tensor, cols: int) -> bool:
    return t.is_cuda and t.dim() == 2 and t.shape[1] == cols and (cols == 1 or t.stride(1) == 1)


def _row_stride(t: torch.Tensor) -> int:
    # the stride of a single row says nothing
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


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
    assert x.dim() == 2 and x.dtype is torch.bfloat16
    T, H = x.shape
    assert _rows_ok(x, H) and _dense(weight, torch.bfloat16, (H,))
    assert residual is None or (residual.dtype is torch.bfloat16 and residual.shape[0] == T
                                and _rows_ok(residual, H))
    assert fmt is None or fmt in _Q_FORMATS
    block = _Q_BLOCK.get(fmt)
    if block and H % block:  # the library's refusal, before a scale buffer of a wrong shape is made
        raise B.MoEError(B.MOE_ERR_UNSUPPORTED, "moe_add_rms_norm")
    if out is None:
        y = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        r = torch.empty_like(y) if residual is not None else None
        q = torch.empty(T, H, dtype=torch.uint8, device=x.device) if fmt else None
        s = torch.empty(T, H // block, dtype=torch.uint8, device=x.device) if block else None
    else:
        y, r, q, s = out
        assert y is None or _dense(y, torch.bfloat16, (T, H))
        assert (r is None) == (residual is None) and (r is None or _dense(r, torch.bfloat16, (T, H)))
        assert (q is None) == (fmt is None) and (q is None or _dense(q, torch.uint8, (T, H)))
        assert (s is None) == (block is None) and (s is None or _dense(s, torch.uint8, (T, H // block)))
    B.moe_add_rms_norm(x.data_ptr(), _row_stride(x), residual.data_ptr() if residual is not None else None,
                       _row_stride(residual) if residual is not None else 0, weight.data_ptr(), eps, T, H,
                       r.data_ptr() if r is not None else None, y.data_ptr() if y is not None else None,
                       q.data_ptr() if q is not None else None, s.data_ptr() if s is not None else None,
                       _Q_FORMATS[fmt] if fmt else 0, scale, _stream_ptr(stream))
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
    scores).  Logits of -inf mask an expert; slots left over get id -1."""
    assert logits.dim() == 2 and logits.dtype in (torch.float32, torch.bfloat16)
    assert scoring in ("softmax", "sigmoid")
    T, E = logits.shape
    assert _rows_ok(logits, E) and (bias is None or _dense(bias, torch.float32, (E,)))
    if out is None:
        idx = torch.empty(T, top_k, dtype=torch.int32, device=logits.device)
        w = torch.empty(T, top_k, dtype=torch.float32, device=logits.device)
    else:
        idx, w = out
        assert _dense(idx, torch.int32, (T, top_k)) and _dense(w, torch.float32, (T, top_k))
    B.moe_topk_route(logits.data_ptr(), logits.dtype is torch.bfloat16, _row_stride(logits),
                     bias.data_ptr() if bias is not None else None, T, E, top_k, scoring == "sigmoid",
                     num_groups, top_groups, renormalize, scale, idx.data_ptr(), w.data_ptr(),
                     _stream_ptr(stream))
    return idx, w


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
        assert _dense(codes, torch.uint8, (rows, cols // 2))
        assert _dense(block_scales, torch.uint8, (rows, cols // 16))
        assert _dense(global_scale, torch.float32, (1,))
        self.rows, self.cols, self.max_tokens = rows, cols, max_tokens
        self.weights = (codes, block_scales, global_scale)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=codes.device)
        self.handle = B.moe_fp4_linear_create(rows, cols, max_tokens, codes.data_ptr(),
                                              block_scales.data_ptr(), global_scale.data_ptr(),
                                              self.workspace.data_ptr(), n, _stream_ptr(stream))

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, *,
                out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """x BF16 [T, cols] (rows may be strided by a multiple of 8) -> [T, rows] in
        out_dtype (bfloat16 or float32) or in `out`'s type."""
        assert x.dtype is torch.bfloat16 and _rows_ok(x, self.cols)
        T = x.shape[0]
        if out is None:
            assert out_dtype in (torch.bfloat16, torch.float32)
            out = torch.empty(T, self.rows, dtype=out_dtype, device=x.device)
        else:
            assert out.dtype in (torch.bfloat16, torch.float32) and _dense(out, out.dtype, (T, self.rows))
        B.moe_fp4_linear(self.handle, x.data_ptr(), _row_stride(x), T, out.data_ptr(),
                         out.dtype is torch.float32, _stream_ptr(stream))
        return out


class Fp4MoELayer(_Fp4Handle):
    """The whole MoE layer for 1..max_tokens (<= 16) tokens on NVFP4 experts, read
    in the checkpoint's layout; same inputs and routes as MegaMoELayer.forward.
    The object keeps the bound weights and its own workspace.  Forwards of one
    object must not overlap on the GPU."""

    def __init__(self, hidden: int, inter: int, num_experts: int, top_k: int, *, max_tokens: int = 16,
                 check_routes: bool = True):
        self.H, self.I, self.E, self.K = hidden, inter, num_experts, top_k
        self.max_tokens = max_tokens
        self.flags = B.MOE_FLAG_CHECK_ROUTES if check_routes else 0
        self._ws_bytes = B.moe_fp4_workspace_query(hidden, inter, num_experts, top_k, self.flags, max_tokens)

    def bind_weights(self, w1, w1_scales, w1_global, w2, w2_scales, w2_global, stream=None) -> None:
        """w1 uint8 [E, 2I, H/2] (gate rows, then up rows) with scales uint8 [E, 2I, H/16]
        and float32 [E]; w2 uint8 [E, H, I/2] likewise."""
        E, H, I = self.E, self.H, self.I
        assert _dense(w1, torch.uint8, (E, 2 * I, H // 2)) and _dense(w2, torch.uint8, (E, H, I // 2))
        assert _dense(w1_scales, torch.uint8, (E, 2 * I, H // 16))
        assert _dense(w2_scales, torch.uint8, (E, H, I // 16))
        assert _dense(w1_global, torch.float32, (E,)) and _dense(w2_global, torch.float32, (E,))
        self.close()
        self.weights = (w1, w1_scales, w1_global, w2, w2_scales, w2_global)
        self.workspace = torch.empty(self._ws_bytes, dtype=torch.uint8, device=w1.device)
        self.handle = B.moe_fp4_create(H, I, E, self.K, self.flags, self.max_tokens,
                                       *(t.data_ptr() for t in self.weights), self.workspace.data_ptr(),
                                       self._ws_bytes, _stream_ptr(stream))

    def forward(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x BF16 [T, H], topk_idx int32 [T, K] (-1: masked slot), topk_w float32 [T, K] -> BF16 [T, H]."""
        if self.handle is None:
            raise B.MoEError(B.MOE_ERR_NOT_BOUND, "moe_fp4_forward")
        T = x.shape[0]
        assert _dense(x, torch.bfloat16, (T, self.H))
        assert _dense(topk_idx, torch.int32, (T, self.K)) and _dense(topk_w, torch.float32, (T, self.K))
        if out is None:
            out = torch.empty(T, self.H, dtype=torch.bfloat16, device=x.device)
        else:
            assert _dense(out, torch.bfloat16, (T, self.H))
        B.moe_fp4_forward(self.handle, x.data_ptr(), topk_idx.data_ptr(), topk_w.data_ptr(), T,
                          out.data_ptr(), _stream_ptr(stream))
        return out
