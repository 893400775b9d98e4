"""Dense products beside the MoE layer, as a user calls them and in plain torch.

Three operators, the parts of a decoder that every token passes:

  linear  x W^T with the layer's FP8 format: E4M3 weights with a power-of-two scale per
          128x128 block, rows of x in E4M3 with one per 128 columns, given as such or
          quantised within the call (serving_route_gb300.Fp8Linear)
  mlp     a gated feed-forward block in BF16 or FP16, y = (act(x Wg^T) * (x Wu^T)) Wd^T,
          the forward (serving_route_gb300.GatedMlp.forward)
  grad    a training step of that block: the forward and the gradients of x and of both
          weights (serving_route_gb300.GatedMlp.forward and .backward)
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through a gate and up projection of the DeepSeek-V3 shape
        {"name": "linear T1 4096x7168", "op": "linear", "T": 1, "rows": 4096, "cols": 7168, "codes": False,
         "f32": False},
        # sixteen tokens (a small batch) through the down projection of that shape
        {"name": "linear T16 7168x2048", "op": "linear", "T": 16, "rows": 7168, "cols": 2048, "codes": False,
         "f32": False},
        # a batch of decoded tokens between the few and a prompt
        {"name": "linear T200 2048x7168", "op": "linear", "T": 200, "rows": 2048, "cols": 7168, "codes": False,
         "f32": False},
        # an odd number of tokens and of rows, float32 out: a head over the V2-Lite expert width
        {"name": "linear T1021 10007x1408 f32", "op": "linear", "T": 1021, "rows": 10007, "cols": 1408,
         "codes": True, "f32": True},
        # a prompt through the gate and up projection, from the norm's 8-bit rows
        {"name": "linear T8192 4096x7168 codes", "op": "linear", "T": 8192, "rows": 4096, "cols": 7168,
         "codes": True, "f32": False},
        # one decoded token through a shared expert of the DeepSeek-V3 shape: its weights' time
        {"name": "mlp T1 H7168 I2048", "op": "mlp", "T": 1, "H": 7168, "I": 2048, "type": "bf16", "act": "silu"},
        # a small odd batch through a block of the V2-Lite shape, FP16 and GELU
        {"name": "mlp T13 H2048 I1408 fp16 gelu", "op": "mlp", "T": 13, "H": 2048, "I": 1408, "type": "fp16",
         "act": "gelu"},
        # ragged in every size: rows, widths that no tile divides
        {"name": "mlp T333 H1000 I2728", "op": "mlp", "T": 333, "H": 1000, "I": 2728, "type": "bf16", "act": "silu"},
        # a prompt through the shared expert
        {"name": "mlp T8192 H7168 I2048", "op": "mlp", "T": 8192, "H": 7168, "I": 2048, "type": "bf16",
         "act": "silu"},
        # a training step of a small block: latency
        {"name": "grad T33 H520 I264", "op": "grad", "T": 33, "H": 520, "I": 264, "type": "bf16", "act": "silu"},
        # an odd number of tokens, the V2-Lite shape, FP16 and GELU
        {"name": "grad T1021 H2048 I1408 fp16 gelu", "op": "grad", "T": 1021, "H": 2048, "I": 1408, "type": "fp16",
         "act": "gelu"},
        # a training step of the shared expert of the V3 shape on 4096 tokens
        {"name": "grad T4096 H7168 I2048", "op": "grad", "T": 4096, "H": 7168, "I": 2048, "type": "bf16",
         "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, step):
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "mlp", "mlp", "grad"))
    if op == "linear":
        return {"op": op, "T": _log(rng, 1, 8192), "rows": _log(rng, 128, 4096 if rng.random() < 0.5 else 10007),
                "cols": _multiple(rng, 256, 7168, 128), "codes": rng.random() < 0.5, "f32": rng.random() < 0.3}
    c = {"op": op, "T": _log(rng, 1, 8192 if op == "mlp" else 4096), "H": _multiple(rng, 256, 7168, 8),
         "I": _multiple(rng, 256, 2728, 8), "type": rng.choice(("bf16", "bf16", "fp16")),
         "act": rng.choice(("silu", "silu", "gelu"))}
    most = 8192 if op == "mlp" else 4096
    c["T"] = min(c["T"], most * 7168 * 2048 // (c["H"] * c["I"]))  # no dearer than the largest listed
    return c


# ---------------------------------------------------------------------------- inputs
def _exponent(amax):
    """The least e in [-127, 127] with amax <= 448 * 2^e, 0 for 0."""
    m, ex = torch.frexp(amax)
    return torch.where(m == 0, 0, torch.where(m > 0.875, ex - 8, ex - 9)).clamp(-127, 127)


def _rows8(x):
    """E4M3 codes (uint8) of float32 rows, and the E8M0 bytes of their scales per 128 columns."""
    b = x.view(x.shape[0], -1, 128)
    e = _exponent(b.abs().amax(-1))
    q = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn)
    return q.view(x.shape).view(torch.uint8), (e + 127).to(torch.uint8)


def _weight8(gen, rows, cols):
    """E4M3 codes [rows, cols] and power-of-two scales [ceil(rows / 128), cols / 128] of a
    matrix of about unit gain whose blocks differ in size."""
    rb, cb = (rows + 127) // 128, cols // 128
    w = torch.randn(rb * 128, cols, device=DEV, generator=gen) / math.sqrt(cols)
    b = w.view(rb, 128, cb, 128)
    b *= torch.exp2(torch.randint(-2, 3, (rb, 1, cb, 1), device=DEV, generator=gen).float())
    e = _exponent(b.abs().amax((1, 3)))
    q = torch.ldexp(b, -e[:, None, :, None]).to(torch.float8_e4m3fn).view(rb * 128, cols)
    return q[:rows].contiguous().view(torch.uint8), torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 6271 + 29)
    c, st = case, {"case": case}
    if c["op"] == "linear":
        T, rows, cols = c["T"], c["rows"], c["cols"]
        st["w"], st["s"] = _weight8(gen, rows, cols)
        x = torch.randn(T, cols, device=DEV, generator=gen)
        x[:, torch.randint(0, cols, (4,), device=DEV, generator=gen)] *= 20.0  # outlier channels
        if c["codes"]:
            st["xq"], st["xs"] = _rows8(x)
        else:
            st["x"] = x.bfloat16()
        st["out"] = torch.empty(T, rows, dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
        if own:
            import serving_route_gb300 as S
            st["handle"] = S.Fp8Linear(st["w"], st["s"], max_tokens=T)
        return st
    T, H, I, t = c["T"], c["H"], c["I"], TYPES[c["type"]]
    st["x"] = torch.randn(T, H, device=DEV, generator=gen).to(t)
    st["w1"] = (torch.randn(2 * I, H, device=DEV, generator=gen) / math.sqrt(H)).to(t)  # gate rows, then up rows
    st["w2"] = (torch.randn(H, I, device=DEV, generator=gen) / math.sqrt(I)).to(t)
    st["y"] = torch.empty(T, H, dtype=t, device=DEV)
    if c["op"] == "grad":
        st["dy"] = (0.25 * torch.randn(T, H, device=DEV, generator=gen)).to(t)
        st["saved"] = torch.empty(T, 2 * I, dtype=torch.float32, device=DEV)  # gate and up, for the backward pass
        st["grads"] = (torch.empty(T, H, dtype=t, device=DEV), torch.empty(2 * I, H, dtype=t, device=DEV),
                       torch.empty(H, I, dtype=t, device=DEV))
    if own:
        import serving_route_gb300 as S
        st["handle"] = S.GatedMlp(st["w1"], st["w2"], max_tokens=T, activation=c["act"])
    return st


# ---------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    c, h = st["case"], st["handle"]
    if c["op"] == "linear":
        if c["codes"]:
            return h.forward_quantized(st["xq"], st["xs"], out=st["out"])
        return h.forward(st["x"], out=st["out"])
    if c["op"] == "mlp":
        return h.forward(st["x"], out=st["y"])
    y = h.forward(st["x"], out=st["y"], saved=st["saved"])
    dx, dw1, dw2 = h.backward(st["dy"], st["x"], st["saved"], out=st["grads"])
    return {"y": y, "dx": dx, "dw1": dw1, "dw2": dw2}


def _act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 0.134145 * g * g)


def _run_plain(st):
    c = st["case"]
    if c["op"] == "linear":
        xq, xs = (st["xq"], st["xs"]) if c["codes"] else _rows8(st["x"].float())
        x = xq.view(torch.float8_e4m3fn).float().view(c["T"], -1, 128)
        x = torch.ldexp(x, xs.int()[..., None] - 127).view(c["T"], -1)
        w = st["w"].view(torch.float8_e4m3fn).float()
        w = w * st["s"].repeat_interleave(128, 1).repeat_interleave(128, 0)[:c["rows"]]
        y = x @ w.t()
        return y if c["f32"] else y.bfloat16()
    t = TYPES[c["type"]]
    x, w1, w2 = st["x"].float(), st["w1"].float(), st["w2"].float()
    g, u = (x @ w1.t()).chunk(2, -1)
    a, da = _act(c["act"], g)
    y = ((a * u) @ w2.t()).to(t)
    if c["op"] == "mlp":
        return y
    dy = st["dy"].float()
    dh = dy @ w2
    dgu = torch.cat((dh * u * da, dh * a), -1)
    return {"y": y, "dx": (dgu @ w1).to(t), "dw1": (dgu.t() @ x).to(t), "dw2": (dy.t() @ (a * u)).to(t)}


# ---------------------------------------------------------------------------- work
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "linear":
        rows, cols = c["rows"], c["cols"]
        b = rows * cols + 4 * ((rows + 127) // 128) * (cols // 128) + T * rows * (4 if c["f32"] else 2)
        return {"bytes": b + T * (cols + cols // 128 if c["codes"] else 2 * cols), "flops": 2 * T * rows * cols}
    H, I = c["H"], c["I"]
    b = 2 * 3 * H * I + 2 * 2 * T * H
    if c["op"] == "mlp":
        return {"bytes": b, "flops": 6 * T * H * I}
    return {"bytes": b + 2 * 2 * T * H + 2 * 3 * H * I, "flops": 18 * T * H * I}


# ---------------------------------------------------------------------------- 64 bits
def _value64(codes):
    """E4M3 values in float64 from the format: sign, four exponent bits (bias 7), three
    mantissa bits."""
    n = codes.to(torch.int32)
    e, m = (n >> 3) & 15, (n & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    return torch.where(n >= 128, -v, v)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "linear":
        if c["codes"]:
            x = _value64(st["xq"]).unflatten(-1, (-1, 128)) * torch.exp2(st["xs"].double() - 127)[..., None]
        else:
            b = st["x"].double().unflatten(-1, (-1, 128))
            s = torch.exp2(torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / 448.0)).clamp(-127, 127))
            x = (b / s).float().to(torch.float8_e4m3fn).view(torch.uint8)  # (exact in float: x has 8 bits)
            x = _value64(x) * s
        w = _value64(st["w"])
        for i in range(st["s"].shape[0]):
            w[128 * i:128 * i + 128] *= st["s"][i].double().repeat_interleave(128)
        return torch.matmul(x.flatten(1), w.t())
    x, w1, w2 = st["x"].double(), st["w1"].double(), st["w2"].double()
    I = c["I"]
    g = torch.matmul(x, w1[:I].t())
    u = torch.matmul(x, w1[I:].t())
    if c["act"] == "silu":
        p = torch.sigmoid(g)
        a, da = g * p, p + g * p * (1 - p)
    else:
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        p = torch.sigmoid(2 * z)  # (1 + tanh z) / 2
        a, da = g * p, p + g * 2 * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    y = torch.matmul(a * u, w2.t())
    if c["op"] == "mlp":
        return y
    dy = st["dy"].double()
    dh = torch.matmul(dy, w2)
    dg, du = dh * u * da, dh * a
    return {"y": y, "dx": torch.matmul(dg, w1[:I]) + torch.matmul(du, w1[I:]),
            "dw1": torch.cat((torch.matmul(dg.t(), x), torch.matmul(du.t(), x))), "dw2": torch.matmul(dy.t(), a * u)}
