"""The dense products on the GPU against float64: Fp8Linear and GatedMlp, their sizes,
strides, types and edges.  Bounds in dense_reference.py."""
import math

import pytest
import torch

from tests import dense_reference as ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def S():
    import __graft_entry__
    __graft_entry__.build()
    import serving_route_gb300 as S
    return S


def rand(*shape, seed=0, dtype=BF, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed * 1000 + sum(shape))
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def weights8(rows, cols, seed=0):
    """Any codes but NaN, and scales over eight octaves."""
    g = torch.Generator("cuda").manual_seed(seed + rows + cols)
    q = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, device="cuda", generator=g)
    q[(q & 127) == 127] = 0x30
    return q, torch.exp2(torch.randint(-8, 1, ((rows + 127) // 128, cols // 128), device="cuda", generator=g).float())


# ---------------------------------------------------------------------------- linear
LINEAR = [(1, 128, 128), (1, 1, 128), (2, 4096, 512), (3, 130, 7168), (8, 1000, 1408), (16, 7168, 2048), (17, 257, 384),
          (31, 512, 640), (33, 4097, 256), (64, 384, 1024), (65, 100, 2176), (100, 2048, 7168), (128, 1408, 2048),
          (129, 129, 1152), (200, 2048, 4096), (256, 256, 128), (257, 640, 896), (384, 10007, 1408), (1021, 300, 2304),
          (2048, 2048, 512), (4100, 136, 256), (700, 8200, 384)]


@pytest.mark.parametrize("T,rows,cols", LINEAR)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear(S, T, rows, cols, dtype):
    codes, scales = weights8(rows, cols)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    x = rand(T, cols, seed=1)
    x[:, ::97] *= 50
    x[0, :128] = 0
    xq, xs = ref.quantize_rows(x)
    want = ref.linear(xq, xs, codes, scales, dtype)
    guard = torch.full((T + 2, rows), 7.0, dtype=dtype, device="cuda")  # rows around the output stay
    out = guard.view(-1)[rows:rows * (T + 1)].view(T, rows)
    ref.check(lin.forward(x, out=out), want, "forward")
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    first = out.clone()
    out.zero_()
    lin.forward_quantized(xq, xs, out=out)
    assert torch.equal(out, first)  # the rows are rounded to the same codes
    assert lin.read_status() == (0, 0)


def test_linear_rounds_rows_like_the_norm(S):
    """x of one block each: all exponents, halves between codes, subnormals, largest values."""
    codes, scales = weights8(256, 256, seed=2)
    x = torch.zeros(64, 256, device="cuda")
    n = torch.arange(128, device="cuda")
    for t in range(64):
        x[t, :128] = (1 + n / 128) * 2.0 ** (4 * t - 130)
        x[t, 128:] = (n - 64) * 2.0 ** (t - 40)
    x[63] = 3.3895313892515355e38
    x = x.bfloat16()
    xq, xs = ref.quantize_rows(x)
    lin = S.Fp8Linear(codes, scales, max_tokens=64)
    eye = torch.zeros(256, 256, dtype=torch.uint8, device="cuda")
    eye.fill_diagonal_(0x38)  # the identity gives the rounded rows themselves
    unit = S.Fp8Linear(eye, torch.ones(2, 2, device="cuda"), max_tokens=64)
    got = unit.forward(x, out_dtype=F32).double()
    want = (ref.e4m3(xq).unflatten(-1, (-1, 128)) * torch.exp2(xs.double() - 127)[..., None]).flatten(1)
    # the last row rounds to 256 * 2^120 = 2^128, past FP32's largest number: infinity
    assert (want[63] == 2.0 ** 128).all() and (got[63] == math.inf).all()
    got, want = got[:63], want[:63]
    normal = want.abs() >= 2.0 ** -126
    assert torch.equal(got[normal], want[normal]) and (got - want).abs().max() <= 2.0 ** -126
    a, b = lin.forward(x), lin.forward_quantized(xq, xs)  # (the last row's sums are no numbers)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and a[:63].isfinite().all()


@pytest.mark.parametrize("T", [3, 40, 300])
def test_linear_strided_rows_and_other_streams(S, T):
    codes, scales = weights8(520, 512, seed=3)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    wide = rand(T, 1024, seed=4)
    x = wide[:, 256:768]
    want = lin.forward(x.contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lin.forward(x, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        got = lin.forward(x)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 16, 60, 130, 600])
def test_linear_nan_and_infinity_stay_in_their_rows(S, T):
    codes, scales = weights8(384, 384, seed=5)
    lin = S.Fp8Linear(codes, scales, max_tokens=T + 2)
    x = rand(T + 2, 384, seed=6)
    want = lin.forward(x)
    x[T // 2, 5] = math.nan
    got = lin.forward(x)
    rows = torch.arange(T + 2, device="cuda") != T // 2
    assert torch.equal(got[rows], want[rows]) and got[T // 2].isnan().any()


@pytest.mark.parametrize("T", [1, 16, 48, 128, 384])
def test_linear_repeats_and_replays(S, T):
    codes, scales = weights8(1000, 2048, seed=7)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    x = rand(T, 2048, seed=8)
    first = lin.forward(x)
    out = torch.empty_like(first)
    for _ in range(5):
        assert torch.equal(lin.forward(x, out=out), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out=out)
    x2 = rand(T, 2048, seed=9)
    want = lin.forward(x2)
    x.copy_(x2)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_linear_of_no_rows(S):
    codes, scales = weights8(64, 128)
    lin = S.Fp8Linear(codes, scales, max_tokens=4)
    assert lin.forward(torch.empty(0, 128, dtype=BF, device="cuda")).shape == (0, 64)


@pytest.mark.parametrize("scale", [0.0, 3.0, -1.0, math.nan, math.inf, 2.0 ** -140])
def test_linear_refuses_scales_that_are_no_powers_of_two(S, scale):
    codes, scales = weights8(256, 256)
    scales[1, 0] = scale
    with pytest.raises(S.binding.MoEError) as e:
        S.Fp8Linear(codes, scales, max_tokens=4)
    assert e.value.status == S.binding.MOE_ERR_BAD_SCALE


def test_linear_takes_the_quantizers_weights(S):
    w = rand(1, 512, 384, dtype=F32, seed=10)
    q, s = S.MegaMoELayer.quantize_weights(w)
    x = rand(50, 384, seed=11)
    xq, xs = ref.quantize_rows(x)
    lin = S.Fp8Linear(q[0], s[0], max_tokens=50)
    ref.check(lin.forward(x), ref.linear(xq, xs, q[0], s[0], BF))


# ---------------------------------------------------------------------------- mlp
MLP = [(1, 8, 8), (1, 2048, 1408), (2, 520, 264), (5, 128, 2728), (13, 2048, 1408), (16, 1000, 136), (17, 264, 520),
       (33, 520, 264), (64, 384, 1024), (65, 512, 128), (100, 1000, 600), (128, 640, 640), (129, 72, 2056), (256, 512, 512),
       (257, 264, 392), (333, 1000, 2728), (700, 2048, 256), (1021, 256, 1408), (2100, 136, 72)]


def mlp_case(S, T, H, I, dtype, act, seed=0):
    w1, w2 = rand(2 * I, H, seed=seed + 1, dtype=dtype, scale=H ** -0.5), rand(H, I, seed=seed + 2, dtype=dtype,
                                                                              scale=I ** -0.5)
    return w1, w2, rand(T, H, seed=seed + 3, dtype=dtype, scale=1.5), S.GatedMlp(w1, w2, max_tokens=T, activation=act)


@pytest.mark.parametrize("T,H,I", MLP)
@pytest.mark.parametrize("dtype,act,saved_type", [(BF, "silu", F32), (HF, "gelu", F32), (BF, "gelu", BF), (HF, "silu", HF)])
def test_mlp(S, T, H, I, dtype, act, saved_type):
    w1, w2, x, mlp = mlp_case(S, T, H, I, dtype, act)
    guard = torch.full((T + 2, H), 7.0, dtype=dtype, device="cuda")
    want = ref.forward(x, w1, w2, act, dtype)
    ref.check(mlp.forward(x, out=guard[1:-1]), want, "forward")
    saved = torch.full((T + 2, 2 * I), 7.0, dtype=saved_type, device="cuda")
    y = mlp.forward(x, saved=saved[1:-1])
    ref.check(y, want, "training forward")
    for t in (guard, saved):
        assert (t[0] == 7).all() and (t[-1] == 7).all()
    saved = saved[1:-1]
    (g, u, _), (tg, tu, _) = ref.gate(x.double(), w1.double(), act)
    gu, tgu = torch.cat((g, u), -1), torch.cat((tg, tu), -1)
    ref.check(saved, (gu, tgu + ref.half_step(gu.abs() + tgu, saved_type)), "saved")

    dy = rand(T, H, seed=5, dtype=dtype, scale=0.25)
    for grad_type in (dtype, F32):
        old = None
        out = [torch.full((n + 2, m), 7.0, dtype=t, device="cuda") for n, m, t in
               ((T, H, dtype), (2 * I, H, grad_type), (H, I, grad_type))]
        if grad_type is F32:
            for t in out[1:]:
                t[1:-1].normal_()
            old = [t[1:-1].clone() for t in out[1:]]
        grads = mlp.backward(dy, x, saved, out=[t[1:-1] for t in out], accumulate=old is not None)
        for n, got, w in zip(("dx", "dw1", "dw2"), grads,
                             ref.backward(dy, x, saved, w1, w2, act, dtype, grad_type, old)):
            ref.check(got, w, n)
        assert all((t[0] == 7).all() and (t[-1] == 7).all() for t in out)
    assert mlp.read_status() == (0, 0)


@pytest.mark.parametrize("T,H,I,act", [(40, 136, 264, "silu"), (300, 264, 136, "gelu")])
def test_mlp_gradients_against_differences(S, T, H, I, act):
    """Directional differences of the float64 block at the kernel's gradients."""
    w1, w2, x, mlp = mlp_case(S, T, H, I, BF, act)
    dy = rand(T, H, seed=6)
    saved = torch.empty(T, 2 * I, device="cuda")
    mlp.forward(x, saved=saved)
    grads = mlp.backward(dy, x, saved)
    tols = ref.backward(dy, x, saved, w1, w2, act, BF, BF)

    def loss(x, w1, w2):
        g, u = (x @ w1.t()).chunk(2, -1)
        return ((ref.act(act, g)[0] * u) @ w2.t() * dy.double()).sum()

    args = [t.double() for t in (x, w1, w2)]
    for i, (grad, (_, tol)) in enumerate(zip(grads, tols)):
        v = rand(*args[i].shape, seed=7 + i, dtype=torch.float64)
        step = 1e-5
        hi, lo = ([t + s * step * v if j == i else t for j, t in enumerate(args)] for s in (1, -1))
        diff = (loss(*hi) - loss(*lo)) / (2 * step)
        # (the saved gate and up are off by FP32 sums, far below the bound of the gradients)
        assert abs(float((grad.double() * v).sum() - diff)) <= float((tol * v.abs()).sum()) + 1e-6 * float(diff.abs())


@pytest.mark.parametrize("T", [1, 9, 70, 300])
def test_mlp_strides_in_place_and_other_streams(S, T):
    w1, w2, _, mlp = mlp_case(S, T, 512, 264, BF, "silu")
    wide = rand(T, 1040, seed=8)
    x = wide[:, 8:520]
    want = mlp.forward(x.contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved, saved2 = (torch.empty(T, 528, dtype=BF, device="cuda") for _ in range(2))
    got = mlp.forward(x, saved=saved, stream=side)
    side.synchronize()
    assert torch.equal(got, mlp.forward(x.contiguous(), saved=saved2)) and torch.equal(saved, saved2)
    dy = rand(T, 1040, seed=9)[:, 520:1032]
    a, b = mlp.backward(dy, x, saved), mlp.backward(dy.contiguous(), x.contiguous(), saved)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    xc = x.contiguous()
    assert torch.equal(mlp.forward(xc, out=xc), want)


@pytest.mark.parametrize("T", [2, 150])
def test_mlp_gradients_one_at_a_time(S, T):
    w1, w2, x, mlp = mlp_case(S, T, 264, 136, BF, "silu")
    saved = torch.empty(T, 272, device="cuda")
    mlp.forward(x, saved=saved)
    dy = rand(T, 264, seed=10)
    full = mlp.backward(dy, x, saved)
    for i in range(3):
        out = [torch.empty_like(t) if i == j else None for j, t in enumerate(full)]
        got = mlp.backward(dy, x, saved, out=out)
        assert torch.equal(got[i], full[i]) and all(t is None for j, t in enumerate(got) if j != i)


def test_mlp_of_no_rows(S):
    w1, w2, _, mlp = mlp_case(S, 4, 64, 32, BF, "silu")
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    saved = torch.empty(0, 64, dtype=F32, device="cuda")
    assert mlp.forward(e, saved=saved).shape == (0, 64)
    dx, dw1, dw2 = mlp.backward(e, e, saved)
    assert dx.shape == (0, 64) and not dw1.any() and not dw2.any()
    ones = [torch.ones(64, 64, device="cuda"), torch.ones(64, 32, device="cuda")]
    mlp.backward(e, e, saved, out=(None, *ones), accumulate=True)
    assert all((t == 1).all() for t in ones)


@pytest.mark.parametrize("T", [1, 16, 100, 300])
def test_mlp_training_step_in_a_graph(S, T):
    """Forward and backward captured, replayed on changed weights and inputs."""
    w1, w2, x, mlp = mlp_case(S, T, 520, 264, BF, "silu")
    saved, dy, y = torch.empty(T, 528, device="cuda"), rand(T, 520, seed=11), torch.empty(T, 520, dtype=BF, device="cuda")
    out = tuple(torch.empty(s, dtype=BF, device="cuda") for s in ((T, 520), (528, 520), (520, 264)))
    mlp.forward(x, out=y, saved=saved)
    mlp.backward(dy, x, saved, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp.forward(x, out=y, saved=saved)
        mlp.backward(dy, x, saved, out=out)
    for seed in (12, 13):
        for t in (w1, w2, x, dy):
            t.copy_(t.roll(seed, 0))
        y2, saved2 = torch.empty_like(y), torch.empty_like(saved)
        mlp.forward(x, out=y2, saved=saved2)
        want = mlp.backward(dy, x, saved2)
        for t in (y, saved, *out):
            t.zero_()
        graph.replay()
        assert torch.equal(y, y2) and torch.equal(saved, saved2) and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [4, 140])
def test_mlp_far_gates(S, act, T):
    """Gates from -1e4 to 1e4: the activations' limits and their derivatives', no NaN."""
    H = I = 136
    w1 = torch.zeros(2 * I, H, device="cuda")
    w1[:I].fill_diagonal_(1.0)
    w1[I:] = 1.0 / H
    w2 = torch.eye(H, I, device="cuda")
    mlp = S.GatedMlp(w1.bfloat16(), w2.bfloat16(), max_tokens=T, activation=act)
    x = torch.linspace(-1, 1, H, device="cuda").sign() * torch.logspace(-4, 4, H, device="cuda")
    x = (x[None] * torch.linspace(0.5, 1, T, device="cuda")[:, None]).bfloat16()
    w1, w2 = w1.bfloat16(), w2.bfloat16()
    saved = torch.empty(T, 2 * I, device="cuda")
    ref.check(mlp.forward(x, saved=saved), ref.forward(x, w1, w2, act, BF))
    dy = rand(T, H, seed=14)
    for got, w in zip(mlp.backward(dy, x, saved), ref.backward(dy, x, saved, w1, w2, act, BF, BF)):
        ref.check(got, w)


@pytest.mark.parametrize("T", [3, 20, 100, 400])
def test_mlp_nan_stays_in_its_row(S, T):
    w1, w2, x, mlp = mlp_case(S, T, 264, 136, BF, "silu")
    want = mlp.forward(x)
    x[T - 2, 3] = math.nan
    got = mlp.forward(x)
    rows = torch.arange(T, device="cuda") != T - 2
    assert torch.equal(got[rows], want[rows]) and got[T - 2].isnan().all()


def test_linear_then_mlp_as_a_decoder_uses_them(S):
    """The norm's 8-bit rows through a linear, its BF16 output through the block, on one stream."""
    T, H, I = 37, 512, 264
    x, res, gain = rand(T, H, seed=15), rand(T, H, seed=16), rand(H, seed=17)
    codes, scales = weights8(H, H, seed=18)
    scales *= 2.0 ** -8
    w1, w2, _, mlp = mlp_case(S, T, H, I, BF, "silu", seed=19)
    lin = S.Fp8Linear(codes, scales, max_tokens=T)
    y, r, q, s = S.add_rms_norm(x, gain, residual=res, fmt="deepseek")
    a = lin.forward_quantized(q, s)
    out = mlp.forward(a)
    ref.check(a, ref.linear(q, s, codes, scales, BF))
    ref.check(out, ref.forward(a, w1, w2, "silu", BF))
