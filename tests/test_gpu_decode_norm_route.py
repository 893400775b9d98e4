"""GPU: moe_add_rms_norm and moe_topk_route against plain float64 forms.

Norm bounds, from the formula: r is exact (one BF16 rounding of a float sum of
two BF16 numbers, which is what torch's own add gives).  y: BF16 rounding 2^-8
relative (8 significant bits), plus the float mean of H squares, the rsqrt and two products, below
2^-14 relative for the widths here.  8-bit: E4M3 keeps 4 significant bits
(2^-4 relative) above its subnormals (half of 2^-9 in units of the scale).
Route bounds: ids must be a valid descending choice of the float64 scores up
to 1e-6 (float scores are within 2^-22 of them), ties by the lowest index;
weights within 2e-6 relative (exp within 2 ulp, sums of at most 1024 terms).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    import __graft_entry__ as ge
    ge.build()
    import serving_route_gb300
    return serving_route_gb300


def rows(gen, T, H, stride=None, offset=0, scale=1.0):
    """BF16 [T, H], rows `stride` apart, starting `offset` elements into an allocation."""
    stride = stride or H
    flat = torch.zeros(offset + T * stride + 8, dtype=torch.bfloat16, device="cuda")
    v = flat[offset:offset + T * stride].view(T, stride)[:, :H]
    v.copy_((torch.randn(T, H, device="cuda", generator=gen) * scale).bfloat16())
    return v


def check_norm(S, x, w, eps, res, fmt, scale=1.0, **kw):
    T, H = x.shape
    want_r = (x.float() + res.float()).bfloat16() if res is not None else None
    base = (want_r if res is not None else x).double()
    y64 = base / (base.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, r, q, s = S.add_rms_norm(x, w, eps, residual=res, fmt=fmt, scale=scale, **kw)
    torch.cuda.synchronize()
    if res is not None:
        assert torch.equal(r, want_r)
    if y is not None:
        assert torch.all((y.double() - y64).abs() <= (2.0**-8 + 2.0**-14) * y64.abs() + 1e-38)
    if fmt is None:
        assert q is None and s is None
        return y, r, q, s
    v = q.view(torch.float8_e4m3fn).double()
    if fmt == "per_tensor":
        assert s is None
        t = (y64 / scale).clamp(-448, 448)
        assert torch.all((v - t).abs() <= (2.0**-4 + 2.0**-10) * t.abs() + 2.0**-10)
        return y, r, q, s
    bl = 128 if fmt == "deepseek" else 32
    amax = y64.view(T, -1, bl).abs().amax(-1)
    e = s.double() - 127
    lo = amax <= 448.0 * torch.exp2(e) * (1 + 2.0**-14)             # it covers the block
    hi = (amax > 448.0 * torch.exp2(e - 1) * (1 - 2.0**-14)) | (e == -127)  # and no smaller one does
    assert torch.all(lo) and torch.all(torch.where(amax == 0, e == 0, hi))
    sc = torch.exp2(e).repeat_interleave(bl, -1)
    assert torch.all((v * sc - y64).abs() <= (2.0**-4 + 2.0**-10) * y64.abs() + 2.0**-10 * sc)
    return y, r, q, s


@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (3, 2048), (153, 7168), (200, 512), (5, 16384),
                                 (160, 16384), (2, 16512), (7, 8320)])
@pytest.mark.parametrize("fmt", [None, "deepseek", "mxfp8", "per_tensor"])
def test_norm_aligned(S, T, H, fmt):
    gen = torch.Generator("cuda").manual_seed(T * 31 + H)
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=gen)).bfloat16()
    for res in (None, rows(gen, T, H, scale=3.0)):
        check_norm(S, rows(gen, T, H), w, 1e-6, res, fmt, scale=0.02)


@pytest.mark.parametrize("T,H,stride,offset", [(1, 1, 1, 0), (4, 7, 7, 0), (3, 100, 104, 0), (3, 1001, 1003, 1),
                                               (170, 96, 96, 0), (2, 33000, 33000, 0), (5, 256, 264, 0),
                                               (5, 256, 260, 0), (5, 256, 256, 3)])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "deepseek", "per_tensor"])
def test_norm_odd_widths_strides_offsets(S, T, H, stride, offset, fmt):
    bl = {"mxfp8": 32, "deepseek": 128}.get(fmt, 1)
    gen = torch.Generator("cuda").manual_seed(T * 37 + H)
    x, res = rows(gen, T, H, stride, offset), rows(gen, T, H, stride + 2, offset)
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=gen)).bfloat16()
    if H % bl:
        with pytest.raises(S.binding.MoEError) as e:
            S.add_rms_norm(x, w, fmt=fmt)
        assert e.value.status == S.binding.MOE_ERR_UNSUPPORTED
        return
    check_norm(S, x, w, 1e-5, None, fmt, scale=0.05)
    check_norm(S, x, w, 1e-5, res, fmt, scale=0.05)


@pytest.mark.parametrize("H", [256, 250])
def test_norm_in_place_and_without_bf16(S, H):
    gen = torch.Generator("cuda").manual_seed(5)
    x, res = rows(gen, 9, H), rows(gen, 9, H)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    fmt = "deepseek" if H % 128 == 0 else "per_tensor"
    y0, r0, q0, s0 = check_norm(S, x, w, 1e-6, res, fmt, scale=0.01)
    x1, res1 = x.clone(), res.clone()
    y, r, q, s = S.add_rms_norm(x1, w, residual=res1, fmt=fmt, scale=0.01,
                                out=(x1, res1, torch.empty_like(q0), None if s0 is None else torch.empty_like(s0)))
    assert torch.equal(y, y0) and torch.equal(r, r0) and torch.equal(q, q0) and (s is None or torch.equal(s, s0))
    assert y.data_ptr() == x1.data_ptr() and r.data_ptr() == res1.data_ptr()
    _, _, q, _ = S.add_rms_norm(x, w, residual=res, fmt=fmt, scale=0.01,
                                out=(None, torch.empty_like(r0), torch.empty_like(q0),
                                     None if s0 is None else torch.empty_like(s0)))
    assert torch.equal(q, q0)


def test_norm_special_rows(S):
    """An all-zero row, a tiny one, one with an infinity and one with a NaN: each
    stays its own affair."""
    H = 256
    gen = torch.Generator("cuda").manual_seed(6)
    x = rows(gen, 6, H)
    x[1] = 0
    x[2] *= 2.0**-100
    x[3, 5], x[4, 7] = math.inf, math.nan
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y, _, q, s = S.add_rms_norm(x, w, 1e-6, fmt="deepseek")
    good = [0, 1, 2, 5]
    yg, _, qg, sg = check_norm(S, x[good].contiguous(), w, 1e-6, None, "deepseek")
    assert torch.equal(y[good], yg) and torch.equal(q[good], qg) and torch.equal(s[good], sg)
    assert not q[1].any() and torch.all(s[1] == 127)
    assert torch.isnan(y[4]).all() and torch.isnan(y[3, 5])


def test_norm_empty_and_refusals(S):
    B = S.binding
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, r, q, s = S.add_rms_norm(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w, fmt="mxfp8")
    assert y.shape == (0, 256) and s.shape == (0, 8)
    x = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(eps=-1.0), dict(eps=math.nan), dict(fmt="per_tensor", scale=0.0),
               dict(fmt="per_tensor", scale=math.inf)):
        with pytest.raises(B.MoEError) as e:
            S.add_rms_norm(x, w, **kw)
        assert e.value.status == B.MOE_ERR_INVALID_ARG
    for bad in (lambda: S.add_rms_norm(x.float(), w), lambda: S.add_rms_norm(x, w[:128]),
                lambda: S.add_rms_norm(x, w, residual=x[:1]), lambda: S.add_rms_norm(x, w, fmt="int8"),
                lambda: S.add_rms_norm(x.t(), w)):
        with pytest.raises(AssertionError):
            bad()


# --------------------------------------------------------------------------- routing
def check_route(S, logits, K, scoring="softmax", bias=None, G=1, TG=1, renorm=True, scale=1.0):
    idx, w = S.topk_route(logits, K, scoring=scoring, bias=bias, num_groups=G, top_groups=TG,
                          renormalize=renorm, scale=scale)
    idx, w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    l = logits.double().cpu().numpy()
    b = np.zeros(l.shape[1]) if bias is None else bias.double().cpu().numpy()
    T, E = l.shape
    gs = E // G
    tol = 1e-6
    for t in range(T):
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                p = 1 / (1 + np.exp(-l[t]))
            c = p + b
        else:
            m = l[t].max()
            p = np.exp(l[t] - m) / np.exp(l[t] - m).sum() if m > -np.inf else np.zeros(E)
            c = l[t].copy()
        free = (l[t] > -np.inf) & (b > -np.inf)
        c = np.where(free, c, -np.inf)
        got = [int(i) for i in idx[t] if i >= 0]
        assert len(set(got)) == len(got) and all(0 <= i < E and free[i] for i in got)
        ok = free.copy()
        if G > 1:
            by = np.sort(c.reshape(G, gs), 1)[:, ::-1]
            if scoring == "sigmoid":
                two = by[:, :2]
                gsc = np.where(np.isfinite(two[:, 0]), np.where(np.isfinite(two), two, 0).sum(1), -np.inf)
            else:
                gsc = by[:, 0]
            order = sorted(range(G), key=lambda g: (-gsc[g], g))[:TG]
            edge = gsc[order[-1]]
            rest = [gsc[g] for g in range(G) if g not in order]
            if rest and edge - max(rest) <= tol and edge != max(rest):
                continue  # too close to call in float
            ok &= np.isin(np.arange(E) // gs, [g for g in order if gsc[g] > -np.inf])
        assert len(got) == min(K, int(ok.sum()))
        assert all(i == -1 for i in idx[t][len(got):]) and all(ok[i] for i in got)
        for a, z in zip(got, got[1:]):
            assert a < z if c[a] == c[z] else c[a] > c[z] - tol
        if got:
            left = [i for i in range(E) if ok[i] and i not in got]
            z = got[-1]
            assert all(i > z if c[i] == c[z] else c[i] < c[z] + tol for i in left)
        want = p[got]
        if renorm and want.sum() > 0:
            want = want / want.sum()
        assert np.allclose(w[t][:len(got)], want * scale, rtol=2e-6, atol=1e-37)
        assert np.all(w[t][len(got):] == 0)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (5, 31, 2), (9, 33, 6), (130, 64, 6), (3, 200, 8),
                                   (2, 512, 32), (2, 1024, 4), (1030, 8, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_softmax(S, T, E, K, dtype):
    gen = torch.Generator("cuda").manual_seed(T + E)
    l = (2 * torch.randn(T, E, device="cuda", generator=gen)).to(dtype)
    check_route(S, l, K)
    check_route(S, l, K, renorm=False, scale=16.0)


@pytest.mark.parametrize("T,E,K,G,TG", [(1, 256, 8, 8, 4), (77, 256, 8, 8, 4), (5, 160, 6, 8, 3), (4, 96, 4, 32, 5),
                                        (6, 60, 2, 20, 1), (3, 24, 4, 3, 3), (2, 1024, 8, 16, 2), (9, 40, 6, 1, 1),
                                        (5, 64, 4, 2, 1), (7, 128, 8, 4, 2), (6, 160, 4, 5, 2), (3, 512, 8, 16, 4),
                                        (2, 1024, 8, 32, 9)])
def test_route_sigmoid_groups(S, T, E, K, G, TG):
    gen = torch.Generator("cuda").manual_seed(T + E + G)
    l = torch.randn(T, E, device="cuda", generator=gen)
    bias = 0.1 * torch.randn(E, device="cuda", generator=gen)
    check_route(S, l, K, "sigmoid", bias, G, TG, scale=2.5)
    check_route(S, l, K, "sigmoid", None, G, TG, renorm=False)
    check_route(S, l, K, "softmax", None, G, TG)


def test_route_ties_and_masks(S):
    E, K = 64, 6
    l = torch.zeros(8, E, device="cuda")
    l[1, 40:44] = 1.0                        # ties above and below the cut
    l[2, ::2], l[2, 1::2] = 0.0, -0.0        # signed zeros are the same choice
    l[3, :] = -math.inf                      # nothing left
    l[4, 3:] = -math.inf                     # three left
    l[5, :] = torch.finfo(torch.float32).min # the type's lowest value is a value
    l[6, :32] = -math.inf
    l[7, 10] = 80.0
    for scoring in ("softmax", "sigmoid"):
        for G, TG in ((1, 1), (4, 2)):
            check_route(S, l, K, scoring, None, G, TG)
    idx, w = S.topk_route(l, K)
    assert idx[0].tolist() == list(range(6)) and idx[2].tolist() == list(range(6))
    assert idx[3].tolist() == [-1] * 6 and not w[3].any()
    assert idx[4].tolist() == [0, 1, 2, -1, -1, -1]
    bias = torch.zeros(E, device="cuda")
    bias[:60] = -math.inf                    # a bias of -inf masks too
    check_route(S, l, K, "sigmoid", bias)


def test_route_nan_rows_are_reported_and_alone(S):
    gen = torch.Generator("cuda").manual_seed(3)
    l = torch.randn(4, 64, device="cuda", generator=gen)
    ref = S.topk_route(l, 4, scoring="sigmoid")
    l[1, 7] = math.nan
    idx, w = S.topk_route(l, 4, scoring="sigmoid")
    assert torch.isnan(w[1]).all() and 7 not in idx[1].tolist()
    for t in (0, 2, 3):
        assert torch.equal(idx[t], ref[0][t]) and torch.equal(w[t], ref[1][t])
    idx, w = S.topk_route(l, 4)
    assert torch.isnan(w[1]).all() and not torch.isnan(w[[0, 2, 3]]).any()


def test_route_strided_rows_streams_and_refusals(S):
    B = S.binding
    gen = torch.Generator("cuda").manual_seed(4)
    wide = torch.randn(50, 100, device="cuda", generator=gen)
    check_route(S, wide[:, :64], 6)
    check_route(S, wide[:, 1:65].bfloat16()[::2], 6)
    want = S.topk_route(wide, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = (torch.empty(50, 4, dtype=torch.int32, device="cuda"), torch.empty(50, 4, device="cuda"))
    torch.cuda.synchronize()
    got = S.topk_route(wide, 4, out=out, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert S.topk_route(wide[:0], 4)[0].shape == (0, 4)
    for kw in (dict(top_k=0), dict(top_k=101), dict(top_k=33), dict(top_k=4, num_groups=3),
               dict(top_k=4, num_groups=50), dict(top_k=4, num_groups=4, top_groups=5),
               dict(top_k=4, bias=torch.zeros(100, device="cuda"))):
        with pytest.raises(B.MoEError) as e:
            S.topk_route(wide, **kw)
        assert e.value.status == B.MOE_ERR_UNSUPPORTED
    for bad in (lambda: S.topk_route(wide.half(), 4), lambda: S.topk_route(wide, 4, scoring="relu"),
                lambda: S.topk_route(wide.t(), 4)):
        with pytest.raises(AssertionError):
            bad()
