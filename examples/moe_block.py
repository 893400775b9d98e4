"""The MoE block of a decoder on one NVFP4 checkpoint: residual norm, expert
choice, routed experts and a shared expert, for a prompt and then token by token.

  python examples/moe_block.py [--tokens 1] [--prompt 2048] [--steps 20] [--small]

Few tokens (up to 16) run on the four-bit weights as they are stored, where
reading them is all the time goes into; a prompt runs on the same weights
requantised once to 128x128 FP8, and its layer takes the norm's 8-bit output as
it is, and its shared expert is one gated feed-forward block.  The few-token step is captured in a CUDA graph.  The weights are random, and
the gate's are in NVFP4 like the others: a checkpoint that keeps its gate in BF16
or float multiplies it by other means (y @ gate.t()), as the prompt does here.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_route_gb300 as S  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def random_fp4(gen, n: int, rows: int, cols: int):
    """n random NVFP4 matrices: codes, E4M3 scales per 16 columns, a power of two each."""
    codes = torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(0x38, 0x40, (n, rows, cols // 16), dtype=torch.uint8, device="cuda", generator=gen)
    return codes, scales, torch.full((n,), 2.0 ** -((cols // 2).bit_length() // 2 + 2), device="cuda")


def dequantize(codes, scales, glob, dtype=torch.float64):
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.tensor(E2M1, dtype=dtype, device=codes.device)[nib & 7] * torch.where(nib >= 8, -1, 1)
    return v * scales.view(torch.float8_e4m3fn).to(dtype).repeat_interleave(16, -1) * glob.to(dtype)[:, None, None]


class MoEBlock:
    FEW = 16

    def __init__(self, hidden: int, inter: int, experts: int, top_k: int, groups: int, top_groups: int,
                 max_prompt: int, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.H, self.I, self.E, self.K = hidden, inter, experts, top_k
        self.route_args = dict(scoring="sigmoid", num_groups=groups, top_groups=top_groups, scale=2.5)
        self.gain = (torch.rand(hidden, device="cuda", generator=gen) + 0.5).bfloat16()
        self.bias = torch.randn(experts, device="cuda", generator=gen) * 0.02
        self.w1, self.w2 = random_fp4(gen, experts, 2 * inter, hidden), random_fp4(gen, experts, hidden, inter)
        self.gate_w = random_fp4(gen, 1, experts, hidden)
        self.shared_w1, self.shared_w2 = random_fp4(gen, 1, 2 * inter, hidden), random_fp4(gen, 1, hidden, inter)

        # few tokens: the checkpoint's own bytes
        self.gate = S.Fp4Linear(*(t[0] for t in self.gate_w[:2]), self.gate_w[2])
        self.up = S.Fp4Linear(*(t[0] for t in self.shared_w1[:2]), self.shared_w1[2])
        self.down = S.Fp4Linear(*(t[0] for t in self.shared_w2[:2]), self.shared_w2[2])
        self.few = S.Fp4MoELayer(hidden, inter, experts, top_k)
        self.few.bind_weights(*self.w1, *self.w2)

        # many tokens: 128x128 FP8 of the experts, BF16 of the small matrices (their
        # values, six significant bits at most, are exact in it)
        self.many = S.MegaMoELayer(hidden, inter, experts, top_k, max_rows=max_prompt, fuse_fc1=True)
        self.many.bind_weights(*S.MegaMoELayer.requantize_weights_nvfp4(*self.w1),
                               *S.MegaMoELayer.requantize_weights_nvfp4(*self.w2))
        self.gate_bf16, up_bf16, down_bf16 = (
            dequantize(*w, dtype=torch.float32)[0].bfloat16()
            for w in (self.gate_w, self.shared_w1, self.shared_w2))
        self.shared = S.GatedMlp(up_bf16, down_bf16, max_tokens=max_prompt)

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """(block output, new residual), BF16 [T, H]."""
        few = x.shape[0] <= self.FEW
        y, r, q, s = S.add_rms_norm(x, self.gain, residual=residual, fmt=None if few else "deepseek")
        logits = self.gate.forward(y, out_dtype=torch.float32) if few else (y @ self.gate_bf16.t()).float()
        idx, w = S.topk_route(logits, self.K, bias=self.bias, **self.route_args)
        out = self.few.forward(y, idx, w) if few else self.many.forward_quantized(q, s, idx, w)
        if not few:
            return out + self.shared.forward(y), r
        g, u = self.up.forward(y).split(self.I, -1)
        return out + self.down.forward(torch.nn.functional.silu(g) * u), r

    def status(self, few: bool):
        if few:
            return self.few.read_status()
        status = self.many.read_status()
        return status if status != (0, 0) else self.shared.read_status()

    def forward_plain(self, x, residual, idx, w):
        """The same in float64, with the experts idx and weights w."""
        r = (x.float() + residual.float()).bfloat16().double()
        y = r * torch.rsqrt(r.pow(2).mean(-1, keepdim=True) + 1e-6) * self.gain.double()

        def expert(v, w1, w2):
            g, u = (v @ dequantize(*w1)[0].t()).split(self.I, -1)
            return (torch.nn.functional.silu(g) * u) @ dequantize(*w2)[0].t()

        out = expert(y, self.shared_w1, self.shared_w2)
        for e in idx.unique().tolist():
            if e >= 0:
                t, k = (idx == e).nonzero(as_tuple=True)
                part = expert(y[t], *([p[e:e + 1] for p in w_] for w_ in (self.w1, self.w2)))
                out.index_add_(0, t, part * w[t, k].double()[:, None])
        return out, r

    def routes(self, x, residual):
        """The experts and weights that forward chooses."""
        few = x.shape[0] <= self.FEW
        y = S.add_rms_norm(x, self.gain, residual=residual)[0]
        logits = self.gate.forward(y, out_dtype=torch.float32) if few else (y @ self.gate_bf16.t()).float()
        return S.topk_route(logits, self.K, bias=self.bias, **self.route_args)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=1, help="tokens of a decode step, 1 to 16")
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--small", action="store_true", help="a small block instead of H 7168, I 2048, E 256")
    a = ap.parse_args()
    if not 1 <= a.tokens <= MoEBlock.FEW:
        ap.error(f"--tokens: 1 to {MoEBlock.FEW}")
    size = (512, 256, 32, 4, 4, 2) if a.small else (7168, 2048, 256, 8, 8, 4)
    block = MoEBlock(*size, max_prompt=a.prompt)
    gen = torch.Generator("cuda").manual_seed(1)
    draw = lambda T: torch.randn(T, block.H, device="cuda", generator=gen).bfloat16()

    def check(x, residual, out, r, what):
        ref, r64 = block.forward_plain(x, residual, *block.routes(x, residual))
        assert torch.equal(r.double(), r64)
        print(f"{what}: relative error {float((out.double() - ref).norm() / ref.norm()):.1e}")

    x, residual = draw(a.prompt), draw(a.prompt)
    out, r = block.forward(x, residual)
    assert block.status(a.prompt <= block.FEW) == (0, 0)
    n = min(a.prompt, 32)
    ref, _ = block.forward_plain(x[:n], residual[:n], *(t[:n] for t in block.routes(x, residual)))
    print(f"prompt of {a.prompt}: relative error {float((out[:n].double() - ref).norm() / ref.norm()):.1e}"
          f" (first {n} tokens)")

    x, residual = draw(a.tokens), draw(a.tokens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(x, residual)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, r = block.forward(x, residual)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    times = []
    for _ in range(a.steps):
        x.copy_(draw(a.tokens)), residual.copy_(r)
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
    assert block.status(True) == (0, 0)
    check(x, residual, out, r, f"decode of {a.tokens}")
    print(f"decode of {a.tokens}: {sorted(times)[len(times) // 2]:.1f} us a step (graph, median of {a.steps})")


if __name__ == "__main__":
    main()
