"""GPU: the example block against its own float64 form, few tokens and many.

Bounds: BF16 y, logits, gate and up of the shared expert and the two outputs
are rounded to 8 bits each (2^-9 relative on average, half an ulp at most
2^-8): below 1% in norm.  A prompt also has the experts' weights and
activations in E4M3 (4 significant bits; errors of products average to a few
percent, and the requantisation of the weights adds as much): below 8%.
"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    import __graft_entry__ as ge
    ge.build()
    from examples.moe_block import MoEBlock
    return MoEBlock(512, 256, 32, 4, 4, 2, max_prompt=300)


@pytest.mark.parametrize("T", [1, 3, 16, 17, 300])
def test_block(block, T):
    gen = torch.Generator("cuda").manual_seed(T)
    x, res = (torch.randn(T, 512, device="cuda", generator=gen).bfloat16() for _ in range(2))
    out, r = block.forward(x, res)
    assert block.status(T <= 16) == (0, 0)
    ref, r64 = block.forward_plain(x, res, *block.routes(x, res))
    assert torch.equal(r.double(), r64)
    assert (out.double() - ref).norm() <= (0.01 if T <= 16 else 0.08) * ref.norm()


def test_command():
    p = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_block.py"), "--small", "--tokens", "2",
                        "--prompt", "64", "--steps", "3"], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    assert "decode of 2" in p.stdout
