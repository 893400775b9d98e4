"""The decode-side operators around the MoE layer, as a user calls them and in plain torch.

Four operators, the steps of one MoE block of a decoder for few tokens:

  norm    residual addition, root-mean-square norm, and the norm's output in
          8 bits with scales beside its BF16 form (serving_route_gb300.add_rms_norm)
  route   gate logits -> expert ids and weights (serving_route_gb300.topk_route)
  linear  products of 1..16 vectors with an NVFP4 matrix (serving_route_gb300.Fp4Linear)
  moe     the whole MoE layer for 1..16 tokens on NVFP4 experts
          (serving_route_gb300.Fp4MoELayer)

NVFP4 is the checkpoint format the package already reads: E2M1 codes, two per
byte along the columns (even column in the low nibble), one E4M3 scale per 16
columns, one float scale per matrix.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of the DeepSeek-V3 shape: latency of the norm before the MoE layer
        {"name": "norm T1 H7168 fp8", "op": "norm", "T": 1, "H": 7168, "fmt": "deepseek", "residual": True},
        # a prefill of that shape: a pure stream of HBM
        {"name": "norm T8192 H7168 fp8", "op": "norm", "T": 8192, "H": 7168, "fmt": "deepseek", "residual": True},
        # an odd number of tokens at the DeepSeek-V2-Lite width, MXFP8, a first layer without a residual
        {"name": "norm T1021 H2048 mxfp8", "op": "norm", "T": 1021, "H": 2048, "fmt": "mxfp8", "residual": False},
        # routing of one decoded token: sigmoid scores, selection bias, 4 of 8 groups, 8 of 256 experts
        {"name": "route T1 E256 sigmoid", "op": "route", "T": 1, "E": 256, "K": 8, "scoring": "sigmoid",
         "groups": 8, "top_groups": 4, "bf16": False},
        # the same for a prefill
        {"name": "route T8192 E256 sigmoid", "op": "route", "T": 8192, "E": 256, "K": 8, "scoring": "sigmoid",
         "groups": 8, "top_groups": 4, "bf16": False},
        # softmax routing of the V2-Lite shape from BF16 logits (ties are common there)
        {"name": "route T4097 E64 softmax", "op": "route", "T": 4097, "E": 64, "K": 6, "scoring": "softmax",
         "groups": 1, "top_groups": 1, "bf16": True},
        # one token through a shared expert's gate and up projection (V3 shape)
        {"name": "linear T1 4096x7168", "op": "linear", "T": 1, "rows": 4096, "cols": 7168, "f32": False},
        # sixteen tokens (a small batch) through its down projection
        {"name": "linear T16 7168x2048", "op": "linear", "T": 16, "rows": 7168, "cols": 2048, "f32": False},
        # an odd number of rows, a ragged width, float32 out: a small head over the V2-Lite expert width
        {"name": "linear T5 10007x1408 f32", "op": "linear", "T": 5, "rows": 10007, "cols": 1408, "f32": True},
        # one decoded token through the V3-shaped MoE layer: 8 experts are read
        {"name": "moe T1 H7168 I2048 E256", "op": "moe", "T": 1, "H": 7168, "I": 2048, "E": 256, "K": 8},
        # three tokens through the V2-Lite-shaped layer
        {"name": "moe T3 H2048 I1408 E64", "op": "moe", "T": 3, "H": 2048, "I": 1408, "E": 64, "K": 6},
        # sixteen tokens through the V3-shaped layer: about 100 experts are read
        {"name": "moe T16 H7168 I2048 E256", "op": "moe", "T": 16, "H": 7168, "I": 2048, "E": 256, "K": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, step, avoid=()):
    while True:
        v = max(lo, min(hi, _log(rng, lo, hi) // step * step))
        if v not in avoid:
            return v


def draw(rng):
    op = rng.choice(("norm", "route", "linear", "linear", "moe", "moe"))
    if op == "norm":
        fmt = rng.choice(("deepseek", "mxfp8", "none"))
        H = _multiple(rng, 256, 7168, {"deepseek": 128, "mxfp8": 32, "none": 1}[fmt], (3072,))
        return {"op": op, "T": _log(rng, 1, 8192), "H": H, "fmt": fmt, "residual": rng.random() < 0.7}
    if op == "route":
        if rng.random() < 0.5:
            groups = rng.choice((1, 4, 8))
            return {"op": op, "T": _log(rng, 1, 8192), "E": groups * rng.randint(8, 32), "K": rng.choice((2, 4, 6, 8)),
                    "scoring": "sigmoid", "groups": groups, "top_groups": max(1, groups // 2), "bf16": False}
        return {"op": op, "T": _log(rng, 1, 8192), "E": rng.randint(8, 256), "K": rng.choice((1, 2, 4, 6, 8)),
                "scoring": "softmax", "groups": 1, "top_groups": 1, "bf16": rng.random() < 0.5}
    if op == "linear":
        cols = _multiple(rng, 256, 7168, 32, (3072,))
        rows = _log(rng, 128, 12000)
        return {"op": op, "T": rng.randint(1, 16), "rows": rows + (rows == 3072), "cols": cols,
                "f32": rng.random() < 0.3}
    E = _log(rng, 8, 256)
    return {"op": op, "T": _log(rng, 1, 16), "H": _multiple(rng, 512, 7168, 128, (3072,)),
            "I": _multiple(rng, 256, 2048, 128, (1536,)), "E": E, "K": rng.choice((1, 2, 4, 6, 8))}


# ---------------------------------------------------------------------------- inputs
def _fp4_matrix(gen, n, rows, cols):
    """NVFP4 weights of about unit gain: uniform codes (rms 2.93), block scales spread over
    three octaves (rms about 70), the float scale bringing the rms to 1/sqrt(cols)."""
    codes = torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device=DEV, generator=gen)
    scales = torch.randint(0x58, 0x70, (n, rows, cols // 16), dtype=torch.uint8, device=DEV, generator=gen)
    glob = (1.0 + 0.25 * torch.rand(n, device=DEV, generator=gen)) / (2.93 * 70.0 * math.sqrt(cols))
    return codes, scales, glob


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    c, st = case, {"case": case}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        x = torch.randn(T, H, device=DEV, generator=gen)
        x[:, torch.randint(0, H, (4,), device=DEV, generator=gen)] *= 20.0  # outlier channels
        st["x"] = x.bfloat16()
        st["residual"] = (4.0 * torch.randn(T, H, device=DEV, generator=gen)).bfloat16() if c["residual"] else None
        st["weight"] = (1.0 + 0.1 * torch.randn(H, device=DEV, generator=gen)).bfloat16()
        y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        r = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if c["residual"] else None
        q = s = None
        if c["fmt"] != "none":
            q = torch.empty(T, H, dtype=torch.uint8, device=DEV)
            s = torch.empty(T, H // _block(c), dtype=torch.uint8, device=DEV)
        st["out"] = (y, r, q, s)
    elif c["op"] == "route":
        T, E = c["T"], c["E"]
        logits = torch.randn(T, E, device=DEV, generator=gen)
        st["logits"] = logits.bfloat16() if c["bf16"] else logits
        st["bias"] = 0.05 * torch.randn(E, device=DEV, generator=gen) if c["scoring"] == "sigmoid" else None
        st["out"] = (torch.empty(T, c["K"], dtype=torch.int32, device=DEV),
                     torch.empty(T, c["K"], dtype=torch.float32, device=DEV))
    elif c["op"] == "linear":
        codes, scales, glob = _fp4_matrix(gen, 1, c["rows"], c["cols"])
        st["codes"], st["scales"], st["glob"] = codes[0], scales[0], glob
        st["x"] = torch.randn(c["T"], c["cols"], device=DEV, generator=gen).bfloat16()
        st["out"] = torch.empty(c["T"], c["rows"], dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
        if own:
            import serving_route_gb300 as S
            st["handle"] = S.Fp4Linear(st["codes"], st["scales"], st["glob"])
    else:
        T, H, I, E, K = (c[k] for k in ("T", "H", "I", "E", "K"))
        st["w1"] = _fp4_matrix(gen, E, 2 * I, H)
        st["w2"] = _fp4_matrix(gen, E, H, I)
        st["x"] = torch.randn(T, H, device=DEV, generator=gen).bfloat16()
        p, idx = torch.softmax(torch.randn(T, E, device=DEV, generator=gen), -1).topk(K, -1)
        st["idx"] = idx.int()
        st["w"] = p / p.sum(-1, keepdim=True)
        st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        if own:
            import serving_route_gb300 as S
            st["handle"] = S.Fp4MoELayer(H, I, E, K, max_tokens=T)
            st["handle"].bind_weights(*st["w1"], *st["w2"])
    return st


def _block(case):
    return 32 if case["fmt"] == "mxfp8" else 128


# ---------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _norm_out(y, r, q, s):
    """Outputs as typed tensors: E4M3 codes and E8M0 scale bytes viewed as the torch types
    whose values they are."""
    out = {"y": y}
    if r is not None:
        out["residual"] = r
    if q is not None:
        out["q"] = q.view(torch.float8_e4m3fn)
        out["scale"] = s.view(torch.float8_e8m0fnu)
    return out


def _run_own(st):
    import serving_route_gb300 as S
    c = st["case"]
    if c["op"] == "norm":
        fmt = None if c["fmt"] == "none" else c["fmt"]
        return _norm_out(*S.add_rms_norm(st["x"], st["weight"], 1e-6, residual=st["residual"], fmt=fmt, out=st["out"]))
    if c["op"] == "route":
        idx, w = S.topk_route(st["logits"], c["K"], scoring=c["scoring"], bias=st["bias"], num_groups=c["groups"],
                              top_groups=c["top_groups"], renormalize=True, scale=2.5, out=st["out"])
        return {"idx": idx, "w": w}
    if c["op"] == "linear":
        return st["handle"].forward(st["x"], out=st["out"])
    return st["handle"].forward(st["x"], st["idx"], st["w"], out=st["out"])


def _run_plain(st):
    c = st["case"]
    if c["op"] == "norm":
        return _plain_norm(c, st["x"], st["residual"], st["weight"])
    if c["op"] == "route":
        return _plain_route(c, st["logits"], st["bias"])
    if c["op"] == "linear":
        w = _dequant(st["codes"], st["scales"], st["glob"])
        y = st["x"].float() @ w.t()
        return y if c["f32"] else y.bfloat16()
    T, K = st["idx"].shape
    e = st["idx"].reshape(-1).long()
    w1 = _dequant(*(t[e] for t in st["w1"]))                                      # [T*K, 2I, H]
    x = st["x"].float().repeat_interleave(K, 0)
    gu = torch.bmm(w1, x[:, :, None])[:, :, 0]
    del w1
    g, u = gu.chunk(2, -1)
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.bmm(_dequant(*(t[e] for t in st["w2"])), h[:, :, None])[:, :, 0]
    return (y.view(T, K, -1) * st["w"][:, :, None]).sum(1).bfloat16()


def _dequant(codes, scales, glob):
    """float32 [..., rows, cols] of NVFP4 parts."""
    lut = torch.tensor(E2M1, device=codes.device)
    pairs = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), -1)            # byte -> (low, high) value
    w = pairs[codes.int()]                                                          # [..., rows, cols/2, 2]
    w = w.view(*scales.shape, 16)
    w *= (scales.view(torch.float8_e4m3fn).float() * glob.view(*glob.shape[:codes.dim() - 2], 1, 1))[..., None]
    return w.flatten(-2)


def _plain_norm(c, x, residual, weight):
    s = x.float()
    r = None
    if residual is not None:
        r = (s + residual.float()).bfloat16()  # the norm is taken of the stored sum
        s = r.float()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * weight.float()
    q = e = None
    if c["fmt"] != "none":
        b = y.view(y.shape[0], -1, _block(c))
        m, ex = torch.frexp(b.abs().amax(-1))
        e = torch.where(m > 0.875, ex - 8, ex - 9)  # the least e with amax <= 448 * 2^e
        e = torch.where(m == 0, 0, e).clamp(-127, 127)
        q = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(y.shape).view(torch.uint8)
        e = (e + 127).to(torch.uint8)
    return _norm_out(y.bfloat16(), r, q, e)


def _plain_route(c, logits, bias):
    l = logits.float()
    T, E = l.shape
    if c["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
        choice = s + bias
    else:
        s = torch.exp(l - l.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
        choice = l
    if c["groups"] > 1:
        by = choice.view(T, c["groups"], -1)
        score = by.sort(dim=-1, descending=True)[0][..., :2].sum(-1)
        keep = score.sort(dim=-1, descending=True, stable=True)[1][:, :c["top_groups"]]
        mask = torch.zeros_like(score, dtype=torch.bool).scatter_(1, keep, True)
        choice = torch.where(mask[..., None], by, -math.inf).view(T, E)
    idx = choice.sort(dim=-1, descending=True, stable=True)[1][:, :c["K"]]              # ties: the lowest index
    w = s.gather(1, idx)
    w = w / w.sum(-1, keepdim=True) * 2.5
    return {"idx": idx.int(), "w": w}


# ---------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        b = 2 * n + 2 * c["H"] + 2 * n + (4 * n if c["residual"] else 0)
        if c["fmt"] != "none":
            b += n + n // _block(c)
        return {"bytes": b, "flops": 6 * n}
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * (2 if c["bf16"] else 4) + 8 * c["K"]), "flops": 8 * c["T"] * c["E"]}
    if c["op"] == "linear":
        mn = c["rows"] * c["cols"]
        return {"bytes": mn * 9 // 16 + c["T"] * (2 * c["cols"] + (4 if c["f32"] else 2) * c["rows"]),
                "flops": 2 * c["T"] * mn}
    T, H, I, E, K = (c[k] for k in ("T", "H", "I", "E", "K"))
    active = E * (1.0 - (1.0 - min(K, E) / E) ** T)  # expected distinct experts of T independent tokens
    return {"bytes": int(active * 3 * H * I * 9 / 16) + 4 * T * H + 8 * T * K, "flops": 6 * T * K * H * I}


# ---------------------------------------------------------------------------- 64 bits
def _value64(codes, scales, glob):
    """NVFP4 values in float64, from the format's definition: sign, two exponent bits
    (bias 1), one mantissa bit; scale sign, four exponent bits (bias 7), three mantissa bits."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    ex, man = (n >> 1) & 3, n & 1
    v = torch.where(ex == 0, man * 0.5, (1.0 + 0.5 * man) * 2.0 ** (ex - 1).double()).double()
    v = torch.where(n >= 8, -v, v)
    s = scales.to(torch.int32)
    se, sm = (s >> 3) & 15, s & 7
    sv = torch.where(se == 0, sm * 2.0 ** -9, (1.0 + sm / 8.0) * 2.0 ** (se - 7).double()).double()
    sv = torch.where(s >= 128, -sv, sv)
    return v * sv.repeat_interleave(16, -1) * glob.double()


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "norm":
        s, res = st["x"].double(), {}
        if st["residual"] is not None:
            r = (s + st["residual"].double()).to(torch.bfloat16)
            res["residual"] = r.double()
            s = r.double()
        y = st["weight"].double() * s / (s.pow(2).sum(-1, keepdim=True) / c["H"] + 1e-6).sqrt()
        res["y"] = y
        if c["fmt"] != "none":
            b = y.unflatten(-1, (-1, _block(c)))
            e = torch.ceil(torch.log2(b.abs().amax(-1) / 448.0)).clamp(-127, 127)
            res["q"] = (b * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).double().flatten(1)
            res["scale"] = torch.exp2(e)
        return res
    if c["op"] == "route":
        l = st["logits"].double()
        p = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.softmax(l, -1)
        pick = p + st["bias"].double() if st["bias"] is not None else p
        if c["groups"] > 1:
            g = pick.unflatten(1, (c["groups"], -1))
            best = g.topk(2, -1)[0].sum(-1).topk(c["top_groups"], -1)[1]
            drop = torch.ones(g.shape[:2], dtype=torch.bool, device=DEV).scatter(1, best, False)
            pick = g.masked_fill(drop[..., None], -math.inf).flatten(1)
        w = p.gather(1, pick.topk(c["K"], -1)[1])
        return {"idx": None, "w": 2.5 * w / w.sum(-1, keepdim=True)}
    if c["op"] == "linear":
        return _value64(st["codes"], st["scales"], st["glob"]).matmul(st["x"].double().t()).t().contiguous()
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
    x, idx = st["x"].double(), st["idx"].tolist()
    for e in sorted({i for row in idx for i in row}):
        at = [(t, k) for t, row in enumerate(idx) for k, i in enumerate(row) if i == e]
        w1 = _value64(*(p[e] for p in st["w1"]))
        w2 = _value64(*(p[e] for p in st["w2"]))
        for t, k in at:
            gate, up = (w1 @ x[t]).split(c["I"])
            out[t] += st["w"][t, k].double() * (w2 @ (torch.sigmoid(gate) * gate * up))
    return out
