"""GPU: the few-token operators on NVFP4 weights against plain float64 forms.

Bounds, from the arithmetic.  Products of a dequantised weight (6 significant
bits) and an activation are exact in float; a float sum of n terms in any order
is within n * 2^-23 of sum |w x| (tensor cores may truncate: one bit more than
rounding), and splits only shorten the chains.  BF16 output: 2^-8 relative.
The layer keeps h in at least 11 significant bits
(2^-11 relative, or 2^-26 of its row's largest); SiLU's exponential and quotient are
within 2^-20.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


@pytest.fixture(scope="module")
def S():
    import __graft_entry__ as ge
    ge.build()
    import serving_route_gb300
    return serving_route_gb300


def fp4(gen, n, rows, cols, lo=0x58, hi=0x70):
    c = torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(lo, hi, (n, rows, cols // 16), dtype=torch.uint8, device="cuda", generator=gen)
    g = (1 + torch.rand(n, device="cuda", generator=gen)) / (200 * math.sqrt(cols))
    return c, s, g


def value64(c, s, g):
    n = torch.stack((c & 15, c >> 4), -1).flatten(-2).long()
    v = E2M1.to(c.device)[n & 7] * torch.where(n >= 8, -1.0, 1.0)
    return v * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * g.double()


def check_linear(S, lin, parts, x, f32):
    w = value64(parts[0], parts[1], parts[2])
    ref = x.double() @ w.t()
    mag = x.double().abs() @ w.abs().t()
    y = lin.forward(x, out_dtype=torch.float32 if f32 else torch.bfloat16)
    assert lin.read_status() == (0, 0)
    n = x.shape[1] / 16 + 32
    bound = n * 2.0**-23 * mag + (0 if f32 else 2.0**-8 * ref.abs() * (1 + 2.0**-8)) + 1e-37
    assert y.dtype == (torch.float32 if f32 else torch.bfloat16) and y.shape == ref.shape
    assert torch.all((y.double() - ref).abs() <= bound)
    return y


@pytest.mark.parametrize("rows,cols", [(1, 32), (31, 64), (33, 512), (64, 96), (130, 1408), (300, 544), (257, 2080),
                                       (4096, 512), (1000, 7168), (5, 16384), (96, 4064), (20011, 128)])
@pytest.mark.parametrize("f32", [False, True])
def test_linear(S, rows, cols, f32):
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    c, s, g = fp4(gen, 1, rows, cols)
    parts = (c[0], s[0], g)
    lin = S.Fp4Linear(*parts)
    for T in (1, 2, 7, 8, 9, 16):
        x = torch.randn(T, cols, device="cuda", generator=gen).bfloat16()
        check_linear(S, lin, parts, x, f32)


def test_linear_every_code_and_scale(S):
    """One row per scale code (NaN codes left out), all E2M1 codes in each block."""
    cols = 256
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")[:128].repeat(254, 1).contiguous()
    codes[:, 1::2] ^= 0x88
    sc = torch.tensor([i for i in range(256) if i & 127 != 127], dtype=torch.uint8, device="cuda")
    s = sc[:, None].repeat(1, cols // 16).contiguous()
    g = torch.tensor([0.125], device="cuda")
    lin = S.Fp4Linear(codes, s, g)
    x = torch.zeros(16, cols, dtype=torch.bfloat16, device="cuda")
    w = value64(codes, s, g)
    for k0 in range(0, cols, 16):          # unit vectors read the matrix back, exactly
        x.zero_()
        for t in range(16):
            x[t, k0 + t] = 1.0
        y = lin.forward(x, out_dtype=torch.float32)
        assert torch.equal(y.double(), w[:, k0:k0 + 16].t())


def test_linear_magnitudes(S):
    """Rows of very different size next to each other: tiny, huge, zero, with an
    outlier; the relative accuracy of each is its own."""
    gen = torch.Generator("cuda").manual_seed(11)
    c, s, g = fp4(gen, 1, 200, 1024)
    parts = (c[0], s[0], g)
    lin = S.Fp4Linear(*parts)
    x = torch.randn(9, 1024, device="cuda", generator=gen)
    x[1] *= 2.0**-90
    x[2] *= 2.0**90
    x[3] = 0
    x[4, 17] = 30000.0
    x[5] = 0
    x[5, 1023] = 2.0**-126
    x[6] *= torch.exp2(torch.randint(-12, 3, (1024,), device="cuda", generator=gen).float())
    x = x.bfloat16()
    check_linear(S, lin, parts, x, True)
    y = check_linear(S, lin, parts, x, False)
    assert not y[3].any()


def test_linear_non_finite_rows_are_alone(S):
    gen = torch.Generator("cuda").manual_seed(12)
    c, s, g = fp4(gen, 1, 100, 512)
    lin = S.Fp4Linear(c[0], s[0], g)
    x = torch.randn(10, 512, device="cuda", generator=gen).bfloat16()
    ref = lin.forward(x).clone()
    x[3, 100], x[6, 511] = math.nan, math.inf
    y = lin.forward(x)
    keep = [t for t in range(10) if t not in (3, 6)]
    assert torch.equal(y[keep], ref[keep])
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[6]).any()


def test_linear_strides_streams_graphs_refusals(S):
    B = S.binding
    gen = torch.Generator("cuda").manual_seed(13)
    c, s, g = fp4(gen, 1, 384, 256)
    parts = (c[0], s[0], g)
    lin = S.Fp4Linear(*parts)
    wide = torch.randn(6, 264, device="cuda", generator=gen).bfloat16()
    check_linear(S, lin, parts, wide[:, 8:], True)
    assert lin.forward(wide[:0, :256]).shape == (0, 384)
    x = wide[:, :256].contiguous()
    want = lin.forward(x)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lin.forward(x, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    gr = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(gr):
        lin.forward(x, out=out)
    for _ in range(3):
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    with pytest.raises(B.MoEError) as e:
        lin.forward(torch.zeros(17, 256, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == B.MOE_ERR_CAPACITY
    for bad in (wide[:, 1:257], torch.zeros(4, 260, dtype=torch.bfloat16, device="cuda")[:, :256]):
        with pytest.raises(B.MoEError) as e:
            lin.forward(bad)
        assert e.value.status == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoEError) as e:
        S.Fp4Linear(c[0, :, :20].contiguous(), s[0], g)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(AssertionError):
        lin.forward(x.float())


def layer64(parts1, parts2, x, idx, w, E, I):
    """(out, sum of magnitudes) in float64."""
    T, H = x.shape
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for t, row in enumerate(idx.tolist()):
        for k, e in enumerate(row):
            if not 0 <= e < E:
                continue
            w1, w2 = value64(*(p[e] for p in parts1)), value64(*(p[e] for p in parts2))
            g, u = (w1 @ x[t].double()).split(I)
            h = g * torch.sigmoid(g) * u
            out[t] += w[t, k].double() * (w2 @ h)
            # |h| with the error of g and u as sums of absolute values
            mag[t] += w[t, k].double().abs() * (w2.abs() @ (h.abs() + 2.0**-26 * h.abs().max()))
    return out, mag


def check_layer(S, parts1, parts2, x, idx, w, layer=None, **kw):
    E, I2, H = parts1[0].shape[0], parts1[0].shape[1], x.shape[1]
    if layer is None:
        layer = S.Fp4MoELayer(H, I2 // 2, E, idx.shape[1], **kw)
        layer.bind_weights(*parts1, *parts2)
    y = layer.forward(x, idx, w)
    assert layer.read_status() == (0, 0)
    ref, mag = layer64(parts1, parts2, x, idx, w, E, I2 // 2)
    # h: 2^-11 rounding, 2^-20 SiLU and the FC1 sums (g and u cancel little here: their
    # float error is below 2^-14 of |h| but where g or u is near zero, where |h| is small)
    bound = 2.0**-8 * (1 + 2.0**-8) * ref.abs() + 2.0**-11 * mag + 1e-37
    assert torch.all((y.double() - ref).abs() <= bound)
    den = ref.norm()
    assert den == 0 or (y.double() - ref).norm() / den <= 2.5e-3
    return y, layer


def routes(gen, T, E, K):
    p, i = torch.softmax(torch.randn(T, E, device="cuda", generator=gen), -1).topk(K, -1)
    return i.int(), (p / p.sum(-1, keepdim=True)).contiguous()


@pytest.mark.parametrize("H,I,E,K", [(128, 128, 1, 1), (512, 256, 8, 2), (256, 1408, 16, 6), (2048, 384, 64, 6),
                                     (1152, 640, 40, 8), (7168, 256, 32, 8), (16384, 128, 4, 2), (128, 16384, 4, 4)])
def test_layer(S, H, I, E, K):
    gen = torch.Generator("cuda").manual_seed(H + I + E)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    layer = None
    for T in (1, 2, 5, 16):
        x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
        y, layer = check_layer(S, p1, p2, x, *routes(gen, T, E, K), layer=layer)
    again = layer.forward(x, *routes(torch.Generator("cuda").manual_seed(1), 16, E, K)).clone()
    for _ in range(5):  # the same bits every time
        assert torch.equal(again, layer.forward(x, *routes(torch.Generator("cuda").manual_seed(1), 16, E, K)))


def test_layer_crowded_experts(S):
    """Every token on the same experts: 16 rows on one expert."""
    H, I, E, K = 1024, 512, 12, 4
    gen = torch.Generator("cuda").manual_seed(21)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    for T in (8, 9, 15, 16):
        idx = torch.tensor([[3, 11, 0, 5]], dtype=torch.int32, device="cuda").repeat(T, 1)
        w = torch.rand(T, K, device="cuda", generator=gen)
        x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
        check_layer(S, p1, p2, x, idx, w)


def test_layer_masked_slots_and_magnitudes(S):
    H, I, E, K = 512, 384, 8, 4
    gen = torch.Generator("cuda").manual_seed(22)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    T = 6
    x = torch.randn(T, H, device="cuda", generator=gen)
    x[3] *= 2.0**-40
    x[4] = 0
    x[5] *= 64
    x = x.bfloat16()
    idx, w = routes(gen, T, E, K)
    idx[0, 1], idx[0, 3], idx[1, :] = -1, -1, -1
    w[0, 1], w[1, 2] = math.nan, math.inf          # masked: ignored
    w[2, 0] = -3.0
    y, layer = check_layer(S, p1, p2, x, idx, w)
    assert not y[1].any() and not y[4].any()
    idx[:] = -1
    y = layer.forward(x, idx, w)
    assert not y.any() and layer.read_status() == (0, 0)


def test_layer_route_errors(S):
    B = S.binding
    H, I, E, K = 256, 128, 8, 2
    gen = torch.Generator("cuda").manual_seed(23)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    x = torch.randn(3, H, device="cuda", generator=gen).bfloat16()
    idx, w = routes(gen, 3, E, K)
    _, layer = check_layer(S, p1, p2, x, idx, w)
    free = S.Fp4MoELayer(H, I, E, K, check_routes=False)
    free.bind_weights(*p1, *p2)
    for change, bit in ((lambda i, v: i.__setitem__((1, 0), 8), B.MOE_DEV_ROUTE_RANGE),
                        (lambda i, v: i.__setitem__((1, 0), -2), B.MOE_DEV_ROUTE_RANGE),
                        (lambda i, v: i.__setitem__((2, 1), int(i[2, 0])), B.MOE_DEV_ROUTE_DUP),
                        (lambda i, v: v.__setitem__((0, 1), math.nan), B.MOE_DEV_ROUTE_NONFINITE)):
        i, v = idx.clone(), w.clone()
        change(i, v)
        layer.forward(x, i, v)
        assert layer.read_status() == (B.MOE_ERR_BAD_ROUTE, bit)
        free.forward(x, i, v)
        assert free.read_status() == ((B.MOE_ERR_BAD_ROUTE, bit) if bit == B.MOE_DEV_ROUTE_RANGE else (0, 0))
    layer.forward(x, idx, w)
    assert layer.read_status() == (0, 0)           # the word is the latest call's


def test_layer_streams_graph_refusals(S):
    B = S.binding
    H, I, E, K = 512, 256, 8, 2
    gen = torch.Generator("cuda").manual_seed(24)
    p1, p2 = fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)
    x = torch.randn(4, H, device="cuda", generator=gen).bfloat16()
    idx, w = routes(gen, 4, E, K)
    want, layer = check_layer(S, p1, p2, x, idx, w, max_tokens=4)
    out = torch.zeros_like(want)
    gr = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, idx, w, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.graph(gr):
        layer.forward(x, idx, w, out=out)
    x2 = torch.randn(4, H, device="cuda", generator=gen).bfloat16()
    i2, w2 = routes(gen, 4, E, K)
    want2, _ = check_layer(S, p1, p2, x2, i2, w2)
    x.copy_(x2), idx.copy_(i2), w.copy_(w2)        # the graph reads the inputs at replay
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)
    assert layer.forward(x[:0], idx[:0], w[:0]).shape == (0, H)
    with pytest.raises(B.MoEError) as e:
        layer.forward(x.repeat(2, 1), idx.repeat(2, 1), w.repeat(2, 1))
    assert e.value.status == B.MOE_ERR_CAPACITY
    unbound = S.Fp4MoELayer(H, I, E, K)
    with pytest.raises(B.MoEError) as e:
        unbound.forward(x, idx, w)
    assert e.value.status == B.MOE_ERR_NOT_BOUND
    for dims in ((100, 256, 8, 2), (512, 100, 8, 2), (512, 256, 8, 3), (512, 256, 0, 2)):
        with pytest.raises(B.MoEError) as e:
            S.Fp4MoELayer(*dims)
        assert e.value.status == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(B.MoEError):
        S.Fp4MoELayer(H, I, E, K, max_tokens=17)
    for bad in (lambda: layer.forward(x.float(), idx, w), lambda: layer.forward(x, idx.long(), w),
                lambda: layer.forward(x, idx[:, :1], w), lambda: layer.bind_weights(*p2, *p1)):
        with pytest.raises(AssertionError):
            bad()


def test_two_layers_in_turn(S):
    """Handles with workspaces of their own do not see each other."""
    H, I, E, K = 384, 256, 6, 2
    gen = torch.Generator("cuda").manual_seed(25)
    sets = [(fp4(gen, E, 2 * I, H), fp4(gen, E, H, I)) for _ in range(2)]
    x = torch.randn(16, H, device="cuda", generator=gen).bfloat16()
    idx, w = routes(gen, 16, E, K)
    ys, layers = zip(*(check_layer(S, *p, x, idx, w) for p in sets))
    for _ in range(3):
        got = [l.forward(x, idx, w) for l in layers]
        assert all(torch.equal(a, b) for a, b in zip(got, ys))
