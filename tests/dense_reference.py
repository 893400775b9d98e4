"""float64 forms of the dense products and bounds on their kernels' errors.

A product's FP32 sum of K terms is off by at most 2 K 2^-24 times the sum of the terms'
magnitudes (rounded or truncated at every step); a rounding to a type by at most
eps / 2 of the value, and in FP16 by 2^-25 below its normal numbers.  The hardware's
exponential and divide in the activations are good to 2^-18 with the factors below.
"""
import math

import torch

U = 2.0 ** -23
FAST = 2.0 ** -18


def half_step(v: torch.Tensor, dtype) -> torch.Tensor:
    r = v.abs() * (torch.finfo(dtype).eps / 2)
    return r + 2.0 ** -25 if dtype is torch.float16 else r


def product(a, b, da=None):
    """a b^T of float64 matrices, and the bound on an FP32 sum of it with a off by da."""
    y = a @ b.t()
    tol = (a.shape[1] * U) * (a.abs() @ b.abs().t())
    if da is not None:
        tol = tol * (1 + U) + da @ b.abs().t()
    return y, tol


def act(name, g):
    """The activation, its derivative, and bounds on the kernels' errors of both."""
    if name == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(z)
    a, d = g * s, s + g * s * torch.sigmoid(-z) * dz
    # exp(-z) is off by about |z| 2^-24 of itself; s (1 - s) |z| < 0.3, and below z = -88 s is 0
    da = FAST * a.abs() + 2.0 ** -22 * g.abs() * s * z.abs() * torch.sigmoid(-z) + 2.0 ** -125 * g.abs()
    return a, d, da, FAST * (1 + g.abs()) * (s + dz * s * torch.sigmoid(-z)) + 2.0 ** -100


def gate(x, w1, name):
    """g, u, h of float64 x and w1, with bounds on the FP32 ones."""
    I = w1.shape[0] // 2
    g, tg = product(x, w1[:I])
    u, tu = product(x, w1[I:])
    a, d, da, _ = act(name, g)
    slope = d.abs() + 0.1  # (|act''| is below 1, and tg far below 0.1)
    return (g, u, a * u), (tg, tu, a.abs() * tu + u.abs() * (da + slope * tg) + slope * tg * tu)


def forward(x, w1, w2, name, dtype):
    _, (_, _, th) = gt = gate(x.double(), w1.double(), name)
    h = gt[0][2]
    y, ty = product(h, w2.double(), th + half_step(h.abs() + th, dtype))
    return y, ty + half_step(y.abs() + ty, dtype)


def backward(dy, x, saved, w1, w2, name, dtype, grad_dtype, old=None):
    """dx, dw1, dw2 from what the forward saved, with bounds; old: what float32 weight
    gradients are added to."""
    dy, x, w1, w2 = (t.double() for t in (dy, x, w1, w2))
    g, u = saved.double().chunk(2, -1)
    dh, tdh = product(dy, w2.t().contiguous())
    a, d, da, dd = act(name, g)
    vals = torch.cat((dh * u * d, dh * a), -1), a * u
    tol = (torch.cat((tdh * (u * d).abs() + dh.abs() * u.abs() * dd + tdh * u.abs() * dd,
                      tdh * a.abs() + dh.abs() * da + tdh * da), -1), u.abs() * da)
    tol = [t + FAST * v.abs() for t, v in zip(tol, vals)]
    tgu, th = (t + half_step(v.abs() + t, dtype) for t, v in zip(tol, vals))
    dgu, h = vals
    out = [product(dgu, w1.t().contiguous(), tgu), product(dgu.t().contiguous(), x.t().contiguous(), tgu.t().contiguous()),
           product(dy.t().contiguous(), h.t().contiguous())]
    out[2] = out[2][0], out[2][1] + dy.abs().t() @ th * (1 + U)
    res = []
    for i, ((v, t), ty) in enumerate(zip(out, (dtype, grad_dtype, grad_dtype))):
        if i and old is not None:
            v = v + old[i - 1].double()
        res.append((v, t + half_step(v.abs() + t, ty)))
    return res


def check(got, want_tol, what=""):
    want, tol = want_tol
    err = (got.double() - want).abs()
    bad = ~(err <= tol + 1e-300)
    assert not bad.any(), (what, int(bad.sum()), float(err.max()), float((err / (tol + 1e-300)).max()),
                           bad.nonzero()[0].tolist())


# ---------------------------------------------------------------------------- FP8
def e4m3(codes):
    """float64 values of E4M3 codes: sign, four exponent bits (bias 7), three mantissa bits."""
    n = codes.to(torch.int32)
    e, m = (n >> 3) & 15, (n & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    v = torch.where((n & 127) == 127, math.nan, v)
    return torch.where(n >= 128, -v, v)


def quantize_rows(x):
    """Codes and E8M0 bytes of float64 rows with a power-of-two scale per 128 columns."""
    b = x.double().unflatten(-1, (-1, 128))
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m == 0, 0, torch.where(m > 0.875, e - 8, e - 9)).clamp(-127, 127)
    q = (b * torch.exp2(-e.double())[..., None]).float().to(torch.float8_e4m3fn)
    return q.flatten(1).view(torch.uint8), (e + 127).to(torch.uint8)


def linear(xq, xs, codes, scales, dtype):
    x = (e4m3(xq).unflatten(-1, (-1, 128)) * torch.exp2(xs.double() - 127)[..., None]).flatten(1)
    s = scales.double().repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)
    y, t = product(x, e4m3(codes) * s)
    return y, t + half_step(y.abs() + t, dtype)
