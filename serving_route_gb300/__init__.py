"""GB300-native single-GPU MoE layer forward (routing -> FP8 quant -> FC1 +
SwiGLU -> FC2 -> combine) behind the C ABI of include/megamoe.h, and the
operators around it for few tokens (norm with 8-bit output, expert choice,
products and the layer on NVFP4 weights), and the dense products beside it
(FP8 linear, gated feed-forward block with its gradients)."""
from . import binding
from .decode import Fp4Linear, Fp4MoELayer, add_rms_norm, topk_route
from .dense import Fp8Linear, GatedMlp
from .layer import MegaMoELayer, sf_atom_rows

__all__ = ["binding", "MegaMoELayer", "sf_atom_rows", "add_rms_norm", "topk_route", "Fp4Linear",
           "Fp4MoELayer", "Fp8Linear", "GatedMlp"]
