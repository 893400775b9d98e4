"""The dense products at their edges on the GPU: refusals of live handles, waits that run
out, offsets past 32 bits, objects side by side on two streams, tiles of every width."""
import math

import pytest
import torch

from tests import dense_reference as ref
from tests.test_gpu_dense import BF, F32, HF, S, mlp_case, rand, weights8  # noqa: F401

pytestmark = pytest.mark.gpu


def status(B, call, *args):
    try:
        call(*args)
    except B.MoEError as e:
        return e.status
    return B.MOE_OK


def test_linear_refusals(S):
    B = S.binding
    codes, scales = weights8(200, 256)
    lin = S.Fp8Linear(codes, scales, max_tokens=8)
    x, out = rand(9, 512, seed=1), torch.zeros(9, 200, dtype=BF, device="cuda")
    xq, xs = torch.zeros(9, 256, dtype=torch.uint8, device="cuda"), torch.zeros(9, 2, dtype=torch.uint8, device="cuda")
    good = dict(x=x.data_ptr(), stride=512, T=8, y=out.data_ptr(), f32=0, stream=0)
    for change, want in ((dict(x=0), "INVALID_ARG"), (dict(x=x.data_ptr() + 2), "INVALID_ARG"), (dict(stride=248), "INVALID_ARG"),
                         (dict(stride=260), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(T=9), "CAPACITY"),
                         (dict(y=0), "INVALID_ARG"), (dict(y=out.data_ptr() + 1), "INVALID_ARG"),
                         (dict(y=out.data_ptr() + 2, f32=1), "INVALID_ARG"), (dict(y=x.data_ptr() + 1024), "INVALID_ARG")):
        assert status(B, B.moe_fp8_linear, lin.handle, *{**good, **change}.values()) == getattr(B, "MOE_ERR_" + want), change
    good = dict(xq=xq.data_ptr(), xs=xs.data_ptr(), T=8, y=out.data_ptr(), f32=0, stream=0)
    for change, want in ((dict(xq=0), "INVALID_ARG"), (dict(xq=xq.data_ptr() + 8), "INVALID_ARG"), (dict(xs=0), "INVALID_ARG"),
                         (dict(T=9), "CAPACITY"), (dict(y=xq.data_ptr()), "INVALID_ARG"), (dict(y=xs.data_ptr()), "INVALID_ARG")):
        assert status(B, B.moe_fp8_linear_quantized, lin.handle, *{**good, **change}.values()) == getattr(B, "MOE_ERR_" + want)
    assert not out.any() and lin.read_status() == (0, 0)


def test_mlp_refusals(S):
    B = S.binding
    w1, w2, _, mlp = mlp_case(S, 8, 64, 32, BF, "silu")
    t = {n: torch.zeros(16, 64, dtype=BF, device="cuda") for n in ("x", "y", "dy", "dx", "dw1", "dw2")}
    saved = torch.zeros(9, 64, device="cuda")
    p = {n: v.data_ptr() for n, v in t.items()}
    good = dict(x=p["x"], stride=64, T=8, y=p["y"], saved=saved.data_ptr(), f32=1, stream=0)
    for change, want in ((dict(x=0), "INVALID_ARG"), (dict(y=0), "INVALID_ARG"), (dict(x=p["x"] + 8), "INVALID_ARG"),
                         (dict(y=p["y"] + 8), "INVALID_ARG"), (dict(saved=saved.data_ptr() + 8), "INVALID_ARG"),
                         (dict(stride=56), "INVALID_ARG"), (dict(stride=68), "INVALID_ARG"), (dict(T=9), "CAPACITY"),
                         (dict(T=-1), "INVALID_ARG"), (dict(y=p["x"] + 128), "INVALID_ARG"), (dict(saved=p["x"]), "INVALID_ARG"),
                         (dict(saved=p["y"]), "INVALID_ARG"), (dict(y=p["x"], stride=128), "INVALID_ARG")):
        assert status(B, B.moe_mlp_forward, mlp.handle, *{**good, **change}.values()) == getattr(B, "MOE_ERR_" + want), change
    good = dict(dy=p["dy"], dys=64, x=p["x"], xs=64, saved=saved.data_ptr(), f32=1, T=8, dx=p["dx"], dw1=p["dw1"],
                dw2=p["dw2"], dwf=0, acc=0, stream=0)
    bad = ["dy", "x", "saved"]
    for change, want in [({n: 0}, "INVALID_ARG") for n in bad] + [({n: p["dx"]}, "INVALID_ARG") for n in bad + ["dw1", "dw2"]] + [
            (dict(dys=60), "INVALID_ARG"), (dict(xs=8), "INVALID_ARG"), (dict(acc=1), "INVALID_ARG"), (dict(T=9), "CAPACITY"),
            (dict(dx=p["dx"] + 8), "INVALID_ARG"), (dict(dw1=p["dw1"] + 8), "INVALID_ARG"), (dict(dw2=p["dw2"] + 4), "INVALID_ARG")]:
        assert status(B, B.moe_mlp_backward, mlp.handle, *{**good, **change}.values()) == getattr(B, "MOE_ERR_" + want), change
    assert not any(v.any() for v in t.values()) and mlp.read_status() == (0, 0)


@pytest.mark.parametrize("T", [1, 40, 2500])
def test_waits_run_out(S, T):
    """A copy that never comes: the calls end, say so, and leave the GPU and the object usable."""
    B = S.binding
    codes, scales = weights8(300, 640, seed=1)
    x = rand(T, 640, seed=2)
    lin = S.Fp8Linear(codes, scales, max_tokens=T, watchdog_test=True)
    for _ in range(2):
        lin.forward(x)
        assert lin.read_status() == (B.MOE_ERR_DEVICE_TIMEOUT, B.MOE_DEV_TIMEOUT)
        assert lin.read_status() == (0, 0)
    w1, w2, xm, mlp = mlp_case(S, T, 264, 136, BF, "silu", seed=3)
    late = S.GatedMlp(w1, w2, max_tokens=T, watchdog_test=True)
    saved = torch.zeros(T, 272, device="cuda")
    late.forward(xm, saved=saved)
    assert late.read_status() == (B.MOE_ERR_DEVICE_TIMEOUT, B.MOE_DEV_TIMEOUT)
    late.backward(xm, xm, saved)
    assert late.read_status() == (B.MOE_ERR_DEVICE_TIMEOUT, B.MOE_DEV_TIMEOUT)
    ref.check(mlp.forward(xm), ref.forward(xm, w1, w2, "silu", BF))
    xq, xs = ref.quantize_rows(x)
    ref.check(S.Fp8Linear(codes, scales, max_tokens=T).forward(x), ref.linear(xq, xs, codes, scales, BF))


def test_linear_offsets_past_32_bits(S):
    """An output of more than 2^31 elements."""
    T, rows, cols = 66000, 33000, 128
    codes, scales = weights8(rows, cols, seed=4)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    x = rand(T, cols, seed=5)
    out = lin.forward(x)
    at = torch.cat((torch.arange(40), torch.arange(T // 2, T // 2 + 40), torch.arange(T - 40, T))).cuda()
    xq, xs = ref.quantize_rows(x[at])
    ref.check(out[at], ref.linear(xq, xs, codes, scales, BF))


def test_mlp_offsets_past_32_bits(S):
    """Saved values and gradients of more than 2^31 elements."""
    T, H, I = 70000, 64, 16384
    w1, w2, x, mlp = mlp_case(S, T, H, I, BF, "silu", seed=6)
    saved = torch.empty(T, 2 * I, device="cuda")
    y = mlp.forward(x, saved=saved)
    at = torch.cat((torch.arange(30), torch.arange(T - 30, T))).cuda()
    ref.check(y[at], ref.forward(x[at], w1, w2, "silu", BF))
    dy = torch.zeros_like(x)
    dy[at] = rand(60, H, seed=7)
    dx, dw1, dw2 = mlp.backward(dy, x, saved)
    want = ref.backward(dy[at], x[at], saved[at], w1, w2, "silu", BF, BF)
    ref.check(dx[at], want[0])
    # the other rows add zeros: the same sums, of more terms for the bound
    ref.check(dw1, want[1])
    ref.check(dw2, want[2])
    assert not dx[30:T - 30].any()


@pytest.mark.parametrize("T", [2, 90, 700])
def test_objects_side_by_side(S, T):
    """Objects on two streams at once, each with its own workspace."""
    sets = []
    for k in range(2):
        codes, scales = weights8(1000, 512, seed=8 + k)
        w1, w2, x, mlp = mlp_case(S, T, 512, 264, BF, "silu", seed=20 * k)
        lin = S.Fp8Linear(codes, scales, max_tokens=T)
        saved = torch.empty(T, 528, device="cuda")
        dy = rand(T, 512, seed=30 + k)
        want = lin.forward(x), mlp.forward(x, saved=saved), *mlp.backward(dy, x, saved)
        sets.append((lin, mlp, x, saved, dy, want))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, (lin, mlp, x, saved, dy, _) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got[k].append((lin.forward(x), mlp.forward(x, saved=saved), *mlp.backward(dy, x, saved)))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for g in got[k] for a, b in zip(g, sets[k][5]))


@pytest.mark.parametrize("T,H,I", [(2304, 320, 8), (2560, 8, 832), (3000, 192, 456), (4096, 64, 704)])
def test_mlp_tiles_of_every_width(S, T, H, I):
    """Many rows of narrow blocks: the pair kernel's tiles of 64, 128, 192 and 256 columns."""
    w1, w2, x, mlp = mlp_case(S, T, H, I, HF, "silu", seed=40)
    saved = torch.empty(T, 2 * I, dtype=HF, device="cuda")
    ref.check(mlp.forward(x, saved=saved), ref.forward(x, w1, w2, "silu", HF))
    dy = rand(T, H, seed=41, dtype=HF, scale=0.1)
    for got, w in zip(mlp.backward(dy, x, saved), ref.backward(dy, x, saved, w1, w2, "silu", HF, HF)):
        ref.check(got, w)


@pytest.mark.parametrize("rows", [63, 190, 193, 450, 1100, 3333, 9000])
@pytest.mark.parametrize("cols", [128, 640, 1664])
def test_linear_tiles_of_every_width(S, rows, cols):
    """2100 tokens: tiles' columns across blocks of the matrix, scale rows of
    every alignment, from views at odd addresses too."""
    T = 2100
    codes, scales = weights8(rows, cols, seed=50)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    xq, xs = ref.quantize_rows(rand(T, cols, seed=51))
    odd = torch.empty(xs.numel() + 3, dtype=torch.uint8, device="cuda")
    for shift in (0, 1, 3):
        s = odd[shift:shift + xs.numel()].view(xs.shape)
        s.copy_(xs)
        ref.check(lin.forward_quantized(xq, s, out_dtype=F32), ref.linear(xq, xs, codes, scales, F32))


def test_linear_values_of_every_code(S):
    """All codes and scales from 2^-127 to 2^127 (products within FP32): exact."""
    codes = torch.zeros(128, 128, dtype=torch.uint8, device="cuda")
    codes.fill_diagonal_(0x38)
    xq = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(1)[:, None].expand(256, 128).contiguous()
    for e in (-127, -100, 0, 30, 100, 127):
        lin = S.Fp8Linear(codes, torch.full((1, 1), 2.0 ** e, dtype=torch.float64, device="cuda").float(), max_tokens=256)
        byte = max(0, min(254, 127 - e))  # the two scales cancel, as far as bytes go
        xs = torch.full((256, 1), byte, dtype=torch.uint8, device="cuda")
        y = lin.forward_quantized(xq, xs, out_dtype=F32).double()
        want = ref.e4m3(xq) * 2.0 ** (e + byte - 127)
        nan = want.isnan()
        # a NaN code makes its whole row one (0 * NaN); the others are single products
        assert torch.equal(y[~nan.any(1)], want[~nan.any(1)]) and y[nan.any(1)].isnan().all()


@pytest.mark.parametrize("T", [1, 7, 16])
@pytest.mark.parametrize("rows,cols", [(4096, 7168), (20000, 3968), (130, 32768), (9000, 16384)])
def test_linear_few_tokens_long_rows(S, T, rows, cols):
    """Many K blocks for each CTA: the ring goes round several times."""
    codes, scales = weights8(rows, cols, seed=60)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    x = rand(T, cols, seed=61)
    xq, xs = ref.quantize_rows(x)
    got = lin.forward(x)
    ref.check(got, ref.linear(xq, xs, codes, scales, BF))
    assert torch.equal(got, lin.forward_quantized(xq, xs))


@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("H,I", [(16384, 4096), (4096, 20000)])
def test_mlp_few_tokens_long_rows(S, T, H, I):
    w1, w2, x, mlp = mlp_case(S, T, H, I, BF, "silu", seed=70)
    ref.check(mlp.forward(x), ref.forward(x, w1, w2, "silu", BF))


@pytest.mark.parametrize("T,rows,cols", [(4911, 136, 128), (6439, 136, 128), (4890, 16, 1536), (2076, 136, 3968),
                                         (6840, 536, 1536), (2585, 784, 128)])
def test_linear_many_tokens_few_rows(S, T, rows, cols):
    """A few tiles of the matrix for dozens of tiles of tokens: narrow pairs, and splits."""
    codes, scales = weights8(rows, cols, seed=80)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    x = rand(T, cols, seed=81)
    xq, xs = ref.quantize_rows(x)
    got = lin.forward(x, out_dtype=F32)
    ref.check(got, ref.linear(xq, xs, codes, scales, F32))
    assert torch.equal(got, lin.forward_quantized(xq, xs, out_dtype=F32))


@pytest.mark.parametrize("T,H,I", [(6498, 128, 264), (4929, 1920, 16), (5014, 1792, 136), (4922, 136, 768), (2454, 16, 2432),
                                   (289, 128, 7936)])
def test_mlp_many_tokens_few_rows(S, T, H, I):
    w1, w2, x, mlp = mlp_case(S, T, H, I, BF, "gelu", seed=90)
    saved = torch.empty(T, 2 * I, device="cuda")
    ref.check(mlp.forward(x, saved=saved), ref.forward(x, w1, w2, "gelu", BF))
    dy = rand(T, H, seed=91, scale=0.1)
    for got, w in zip(mlp.backward(dy, x, saved), ref.backward(dy, x, saved, w1, w2, "gelu", BF, BF)):
        ref.check(got, w)


def test_outputs_that_overlap_the_weights_are_refused(S):
    B = S.binding
    codes, scales = weights8(256, 256, seed=3)
    kept = codes.clone()
    lin = S.Fp8Linear(codes, scales, max_tokens=8)
    x = rand(8, 256, seed=4)
    xq, xs = ref.quantize_rows(x)
    inside = codes.data_ptr() + 4096
    assert status(B, B.moe_fp8_linear, lin.handle, x.data_ptr(), 256, 8, inside, 0, 0) == B.MOE_ERR_INVALID_ARG
    assert status(B, B.moe_fp8_linear_quantized, lin.handle, xq.data_ptr(), xs.data_ptr(), 8, inside, 0,
                  0) == B.MOE_ERR_INVALID_ARG
    assert torch.equal(codes, kept)
    w1, w2, xm, mlp = mlp_case(S, 8, 64, 32, BF, "silu", seed=5)
    kept = w1.clone(), w2.clone()
    saved, y = torch.zeros(8, 64, device="cuda"), torch.zeros(64, 64, dtype=BF, device="cuda")
    for w in (w1, w2):
        p = w.data_ptr()
        assert status(B, B.moe_mlp_forward, mlp.handle, xm.data_ptr(), 64, 8, p, 0, 0, 0) == B.MOE_ERR_INVALID_ARG
        assert status(B, B.moe_mlp_forward, mlp.handle, xm.data_ptr(), 64, 8, y.data_ptr(), p, 0, 0) == B.MOE_ERR_INVALID_ARG
        for out in ((p, 0, 0), (0, p, 0), (0, 0, p)):
            assert status(B, B.moe_mlp_backward, mlp.handle, xm.data_ptr(), 64, xm.data_ptr(), 64, saved.data_ptr(), 1, 8,
                          *out, 0, 0, 0) == B.MOE_ERR_INVALID_ARG
    assert torch.equal(w1, kept[0]) and torch.equal(w2, kept[1]) and mlp.read_status() == (0, 0)
