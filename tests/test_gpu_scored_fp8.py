"""Scored routing and the 8-bit floating point operators on the GPU against 64-bit references.

Half a step of a type, relative to the value: H(t) = finfo(t).eps / 2 (fp32 2^-24, BF16 2^-8, E4M3 2^-4).  Each
tolerance below is counted in such steps, from the roundings of the formula it checks."""
import numpy as np
import pytest
import torch

import quantized_grouped_gemm_amd as qgg

from .gpu_util import DEV

pytestmark = pytest.mark.gpu

H32, HBF = 2.0 ** -24, 2.0 ** -8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


# ------------------------------------------------------------------ routing

def scores64(l, score):
    l = l.double()
    fine = torch.isfinite(l)
    l = torch.where(fine, l, torch.full_like(l, -np.inf))
    if score == "sigmoid":
        s = torch.special.expit(l)
    else:
        m = l.amax(1, keepdim=True)
        s = torch.exp(l - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
        z = s.sum(1, keepdim=True)
        s = torch.where(z > 0, s / z, torch.zeros_like(s))
    return torch.where(fine, s, torch.zeros_like(s)), fine


def route64(l, k, score, bias, n_group, topk_group, group_top, renorm, scale):
    s, fine = scores64(l, score)
    c = s + (0 if bias is None else torch.nan_to_num(bias.double(), nan=0, posinf=0, neginf=0))
    c = torch.where(fine, c, torch.full_like(c, -np.inf))
    if bias is not None:
        c[:, ~torch.isfinite(bias)] = -np.inf
    T, E = c.shape
    size = E // n_group
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        v = c[t].numpy()
        pool = list(range(E))
        if topk_group < n_group:
            gs = [np.sort(v[j * size:(j + 1) * size])[::-1][:group_top].sum() for j in range(n_group)]
            kept = sorted(range(n_group), key=lambda j: (-gs[j], j))[:topk_group]
            pool = [e for e in pool if e // size in kept]
        ids[t] = sorted(pool, key=lambda e: (-v[e], e))[:k]
    ids = torch.from_numpy(ids)
    w = torch.gather(s, 1, ids.long())
    if renorm:
        z = w.sum(1, keepdim=True)
        w = torch.where(z > 0, w / z, torch.zeros_like(w))
    return ids, w * scale


ROUTE = [
    dict(T=1, E=1, k=1), dict(T=3, E=64, k=8), dict(T=65, E=197, k=7), dict(T=130, E=256, k=8, n_group=8, topk_group=4),
    dict(T=33, E=384, k=8, n_group=8, topk_group=3, group_top=1), dict(T=9, E=1024, k=32, n_group=64, topk_group=33),
    dict(T=21, E=160, k=6, n_group=5, topk_group=2), dict(T=17, E=64, k=4, n_group=64, topk_group=7, group_top=1),
    dict(T=40, E=513, k=2, n_group=27, topk_group=4),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("c", ROUTE, ids=lambda c: f"T{c['T']}E{c['E']}k{c['k']}g{c.get('n_group', 1)}")
def test_route_scored(c, score, renorm):
    c = dict(dict(n_group=1, topk_group=1, group_top=2), **c)
    if c["n_group"] == 1:
        c["group_top"] = 1
    g = gen(c["T"] * 1000 + c["E"])
    for dtype in (torch.float32, torch.bfloat16):
        l = normal(g, c["T"], c["E"], std=2.0, dtype=dtype)
        for bias in (None, normal(g, c["E"], std=0.05, dtype=torch.float32)):
            a = (c["k"], score, bias, c["n_group"], c["topk_group"], c["group_top"], renorm, 2.5)
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            ids, gates = qgg.moe_route_scored(l.to(DEV), a[0], score, None if bias is None else bias.to(DEV), *a[3:],
                                              err_flag=err)
            rid, rg = route64(l, *a)
            assert torch.equal(ids.cpu(), rid)
            # 64-bit arithmetic, one rounding to fp32
            assert torch.all((gates.cpu().double() - rg).abs() <= 1.01 * H32 * rg.abs() + 1e-44)
            assert err.item() == 0


def test_route_ties_go_to_the_lower_id():
    # equal logits everywhere; then equal pairs; then equal groups
    for n_group, topk_group in ((1, 1), (4, 2)):
        l = torch.zeros(2, 64, device=DEV)
        ids, gates = qgg.moe_route_scored(l, 6, "sigmoid", None, n_group, topk_group, 2, True, 1.0)
        assert ids.cpu().tolist() == [list(range(6))] * 2
        assert torch.all((gates.cpu().double() - 1 / 6).abs() <= 1.01 * H32 / 6)
    l = torch.arange(128, device=DEV).float().flip(0).div(2).floor().repeat(3, 1) / 16
    ids, _ = qgg.moe_route_scored(l, 9, "softmax")
    assert ids.cpu().tolist() == [list(range(9))] * 3
    # a bias that makes two different scores equal leaves the id order to decide
    l = torch.full((1, 256), -2.0, device=DEV)
    bias = torch.zeros(256, device=DEV)
    bias[200] = bias[70] = bias[71] = 0.25
    ids, _ = qgg.moe_route_scored(l, 4, "sigmoid", bias)
    assert ids.cpu().tolist() == [[70, 71, 200, 0]]


def test_route_keeps_scores_apart_that_fp32_would_merge():
    # sigmoid(17) and sigmoid(18) round to the same fp32 number (1 - 4e-8, 1 - 1.5e-8)
    l = torch.linspace(17.0, 18.0, 64, device=DEV).repeat(2, 1).contiguous()
    ids, _ = qgg.moe_route_scored(l, 8, "sigmoid")
    assert ids.cpu().tolist() == [list(range(63, 55, -1))] * 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group", [(60, 1, 1), (256, 8, 3), (384, 1, 1)])
def test_route_choices_that_fp32_cannot_make(score, E, n_group, topk_group):
    """A bias that takes nearly all of each score away: the choice values differ by parts in 10^8, and order as in
    64 bits (whose own rounding is 10^8 times smaller).  Near logits without a bias, large and small ones likewise."""
    g = gen(E)
    l = normal(g, 50, E, std=1.0, dtype=torch.float32)
    l[:] = l[0]                                  # one bias for all rows
    l += (torch.rand(50, E, generator=g) - 0.5) * 2e-6
    bias = -scores64(l[:1], score)[0][0].float()
    near = normal(g, 50, 1, std=1.0, dtype=torch.float32) + torch.rand(50, E, generator=g) * 1e-6
    far = torch.where(torch.rand(50, E, generator=g) < 0.5, 22.0, -640.0) + torch.rand(50, E, generator=g) * 15
    for x, b in ((l, bias), (near, None), (far, None), (far, bias), (near, bias)):
        for top in (1, 2):
            a = (6, score, b, n_group, topk_group, top, True, 1.0)
            ids, gates = qgg.moe_route_scored(x.to(DEV), 6, score, None if b is None else b.to(DEV), *a[3:])
            rid, rg = route64(x, *a)
            assert torch.equal(ids.cpu(), rid)
            assert torch.all((gates.cpu().double() - rg).abs() <= 1.01 * H32 * rg.abs() + 1e-44)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_values_that_are_not_finite(score):
    g = gen(5)
    l = normal(g, 6, 96, dtype=torch.float32)
    l[0, :] = -np.inf                       # nothing left
    l[1, 3:] = -np.inf                      # fewer than k left
    l[2, 5] = np.nan
    l[3, 7] = np.inf
    l[4, :] = torch.finfo(torch.float32).min
    bias = normal(g, 96, std=0.1, dtype=torch.float32)
    bias[11] = -np.inf
    bias[12] = np.nan
    for n_group, topk_group in ((1, 1), (4, 2)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ids, gates = qgg.moe_route_scored(l.to(DEV), 8, score, bias.to(DEV), n_group, topk_group, 2, True, 1.0,
                                          err_flag=err)
        rid, rg = route64(l, 8, score, bias, n_group, topk_group, 2, True, 1.0)
        assert torch.equal(ids.cpu(), rid)
        assert torch.all((gates.cpu().double() - rg).abs() <= 1.01 * H32 * rg.abs() + 1e-44)
        assert err.item() & 1
        assert torch.all(gates[0] == 0)


def bwd64(l, ids, dg, score, renorm, scale):
    s, _ = scores64(l, score)
    T, E = s.shape
    ok = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1).long()
    u = torch.where(ok, torch.gather(s, 1, at), torch.zeros(1, dtype=torch.float64))
    fine = ok & torch.isfinite(torch.gather(l.double(), 1, at))
    dg = torch.where(fine, dg.double(), torch.zeros(1, dtype=torch.float64))
    if renorm:
        z = u.sum(1, keepdim=True)
        z = torch.where(z > 0, z, torch.ones_like(z))
        du = (dg - (dg * u).sum(1, keepdim=True) / z) / z
    else:
        du = dg
    du = torch.where(fine, du * scale, torch.zeros(1, dtype=torch.float64))
    ds = torch.zeros_like(s).scatter_add_(1, at, du)
    if score == "sigmoid":
        return ds * s * torch.special.expit(-torch.nan_to_num(l.double(), nan=-np.inf, posinf=-np.inf))
    return s * (ds - (ds * s).sum(1, keepdim=True))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 64, 8), (67, 197, 7), (130, 256, 8), (9, 1024, 32), (31, 513, 3)])
def test_route_scored_bwd(T, E, k, score, renorm):
    g = gen(T + E)
    for dtype, h in ((torch.float32, H32), (torch.bfloat16, HBF)):
        l = normal(g, T, E, std=2.0, dtype=dtype)
        ids = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :k].to(torch.int32)
        if T > 4:
            ids[1, 0] = -1
            ids[2, 0] = E                   # outside
            ids[3, 1] = ids[3, 0]           # the same expert twice
        dg = normal(g, T, k, dtype=torch.float32)
        out = qgg.moe_route_scored_bwd(l.to(DEV), ids.to(DEV), dg.to(DEV), score, renorm, 2.5).cpu().double()
        ref = bwd64(l, ids, dg, score, renorm, 2.5)
        # kept forms: 64 bits, rounded when put into the row, by the scale and by the type; subtractions in 64 bits.
        # dense softmax in fp32: exp's argument (up to 20 in size: 20 steps), exp and division (4), sums over E (10 + 6)
        # and over k (6), products (4): 50 steps of what is added, p (|dg| + <|dg|, p>).
        dense = score == "softmax" and not renorm
        s, _ = scores64(l, score)
        spread = torch.zeros_like(s).scatter_add_(1, ids.clamp(0, E - 1).long(), dg.abs().double())
        size = 2.5 * s * (spread + (spread * s).sum(1, keepdim=True)) if dense else 0
        tol = (3 * H32 + (h if dtype == torch.bfloat16 else 0)) * ref.abs() + 50 * H32 * size * (2 if dense else 0) + 1e-14
        assert torch.all((out - ref).abs() <= tol), (out - ref).abs().max()
        kept = torch.zeros(T, E + 1, dtype=torch.bool).scatter_(1, torch.where((ids < 0) | (ids > E), E, ids).long(), True)
        if not dense:
            assert torch.all(out[~kept[:, :E]] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_by_differences(score, renorm):
    # L = <dg, gates>; central differences of the 64-bit forward with the choice fixed, step 1e-4: error ~ 1e-8
    g = gen(11)
    l = normal(g, 3, 24, dtype=torch.float32)
    ids, _ = qgg.moe_route_scored(l.to(DEV), 5, score, renorm=renorm, scale=1.5)
    dg = normal(g, 3, 5, dtype=torch.float32)
    got = qgg.moe_route_scored_bwd(l.to(DEV), ids, dg.to(DEV), score, renorm, 1.5).cpu().double()
    ids = ids.cpu().long()

    def loss(x):
        s = torch.special.expit(x) if score == "sigmoid" else torch.softmax(x, 1)
        w = torch.gather(s, 1, ids)
        w = w / w.sum(1, keepdim=True) if renorm else w
        return (1.5 * w * dg.double()).sum()

    for t in range(3):
        for e in range(24):
            d = torch.zeros(3, 24, dtype=torch.float64)
            d[t, e] = 1e-4
            diff = (loss(l.double() + d) - loss(l.double() - d)) / 2e-4
            assert abs(diff - got[t, e]) <= 2e-6


def test_route_scored_bwd_rows_without_finite_logits():
    l = torch.full((2, 64), -np.inf, device=DEV)
    l[1, 4] = 1.0
    ids = torch.tensor([[0, 1], [4, 9]], dtype=torch.int32, device=DEV)
    dg = torch.ones(2, 2, device=DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            out = qgg.moe_route_scored_bwd(l, ids, dg, score, renorm, 1.0).cpu()
            assert torch.isfinite(out).all()
            assert torch.all(out[0] == 0)


# ------------------------------------------------------------------ 8-bit rows

def e4m3(v):
    """The nearest E4M3 value, ties to even, in 64 bits."""
    _, ex = np.frexp(v)
    step = np.exp2(np.maximum(ex - 1, -6).astype(np.float64) - 3)
    return np.round(v / step) * step


def quantize64(x):
    """(values of the codes, scales) of rows x, in 64 bits."""
    x = np.asarray(x, np.float64)
    M, C = x.shape
    nb = -(-C // 128)
    q, s = np.zeros_like(x), np.ones((M, nb))
    for b in range(nb):
        part = x[:, b * 128:(b + 1) * 128]
        fine = np.isfinite(part)
        top = np.where(fine, np.abs(part), 0).max(1)
        m, ex = np.frexp(top)
        e = np.where(top > 0, np.maximum(np.where(m <= 0.875, ex - 9, ex - 8), -127), 0)
        s[:, b] = np.exp2(e.astype(np.float64))
        with np.errstate(invalid="ignore"):
            q[:, b * 128:(b + 1) * 128] = np.where(fine, e4m3(np.where(fine, part, 0) / s[:, b:b + 1]), np.nan)
    return q, s


def value(codes, scales):
    c, s = codes.cpu().double().numpy(), scales.cpu().double().numpy()
    return c * np.repeat(s, 128, axis=1)[:, :c.shape[1]]


def rows_with_edges(g, M, C):
    x = normal(g, M, C)
    edges = [0.0, -0.0, 448.0, 449.0, 3.3e38, -3.3e38, 1e-38, 9.2e-41, -9.2e-41, float("inf"), float("-inf"), float("nan")]
    for r in range(M):
        x[r] *= 2.0 ** ((r % 9) * 6 - 24)
        x[r, (r * 7) % C] = edges[r % len(edges)]
        if r % 11 == 3:
            x[r] = 0
        if r % 13 == 5:
            x[r] = torch.tensor(9.2e-41)
        if r % 17 == 6:
            x[r] = float("nan")
    return x


@pytest.mark.parametrize("M,C", [(1, 8), (1, 128), (37, 136), (64, 200), (257, 1024), (3, 7168), (50, 2048 + 64)])
def test_quantize_and_back(M, C):
    x = rows_with_edges(gen(M * C), M, C)
    codes, scales = qgg.fp8_quantize(x.to(DEV))
    assert codes.dtype == torch.float8_e4m3fn and scales.dtype == torch.float8_e8m0fnu
    q, s = quantize64(x.double().numpy())
    np.testing.assert_array_equal(scales.cpu().double().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().double().numpy(), q)
    back = qgg.fp8_dequantize(codes, scales).cpu()
    np.testing.assert_array_equal(back.double().numpy(), torch.from_numpy(value(codes, scales)).to(torch.bfloat16).double().numpy())
    # the format's promise: half a step of E4M3, or of its subnormal grid
    fine = torch.isfinite(x).numpy()
    top = np.repeat(s, 128, 1)[:, :C]
    err = np.abs(value(codes, scales) - x.double().numpy())
    assert np.all(err[fine] <= np.maximum(2.0 ** -4 * np.abs(x.double().numpy()), 2.0 ** -10 * top)[fine])


def test_quantize_every_scale_and_every_code():
    # all E4M3 codes times every power of two BF16 holds come back as they are
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7F) != 0x7F].view(torch.float8_e4m3fn).double()
    for e in (-118, -60, -1, 0, 7, 100, 119):
        x = (codes * 2.0 ** e).to(torch.bfloat16).repeat(1, 2)[:, :256].contiguous().view(1, -1)[:, :256]
        x = torch.cat([x[:, :127], torch.full((1, 1), 448.0 * 2.0 ** e, dtype=torch.bfloat16), x[:, 127:254],
                       torch.full((1, 1), -448.0 * 2.0 ** e, dtype=torch.bfloat16)], 1).contiguous()
        c, s = qgg.fp8_quantize(x.to(DEV))
        assert np.all(s.cpu().double().numpy() == 2.0 ** e)
        np.testing.assert_array_equal(value(c, s), x.double().numpy())


def test_dequantize_every_scale():
    """Every scale byte: 2^(c - 127), rounded once to BF16 with the code; 255 is NaN."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 2).contiguous()
    back = qgg.fp8_dequantize(codes.to(DEV), scales.to(DEV)).cpu()
    s = np.exp2(np.arange(256) - 127.0)
    s[255] = np.nan
    want = codes.view(torch.float8_e4m3fn).double() * torch.from_numpy(s)[:, None]
    np.testing.assert_array_equal(back.double().numpy(), want.to(torch.bfloat16).double().numpy())


def test_rows_past_32_bit_offsets():
    M, C = 600_000, 7168                    # 4.3e9 values
    x = torch.empty((M, C), dtype=torch.bfloat16, device=DEV)
    x.normal_()
    x[-5:] *= 1000
    codes, scales = qgg.fp8_quantize(x)
    for lo in (0, M // 2, M - 7):
        c, s = qgg.fp8_quantize(x[lo:lo + 7].contiguous())
        assert torch.equal(c.view(torch.uint8), codes[lo:lo + 7].view(torch.uint8))
        assert torch.equal(s.view(torch.uint8), scales[lo:lo + 7].view(torch.uint8))
    del x
    back = qgg.fp8_dequantize(codes, scales)
    assert torch.equal(back[-7:], qgg.fp8_dequantize(codes[-7:].contiguous(), scales[-7:].contiguous()))


# ------------------------------------------------------------------ SwiGLU

def check_rows(got, want, slack):
    """8-bit rows got = (codes, scales) against 64-bit values known to `slack` (absolute)."""
    v, s = value(*got), got[1].cpu().double().numpy()
    C = v.shape[1]
    top = np.repeat(s, 128, 1)[:, :C]
    err = np.abs(v - want)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * top) + 1.1 * slack), err.max()
    for b in range(s.shape[1]):
        part, sl = np.abs(want[:, b * 128:(b + 1) * 128]), slack[:, b * 128:(b + 1) * 128]
        hi, lo = (part + sl).max(1), (part - sl).max(1)
        live = lo > 0
        assert np.all(lo[live] <= 448 * s[live, b]) and np.all((hi[live] > 224 * s[live, b]) | (s[live, b] == 2.0 ** -127))


def check_exact(got, want):
    """8-bit rows that are those of the 64-bit values: the same scales and codes.  A 64-bit value carries a few times 2^-53,
    and may round another way where it is that near to a border: one value in 2^53 / 2^6, so none is let off."""
    q, s = quantize64(want)
    np.testing.assert_array_equal(got[1].cpu().double().numpy(), s)
    np.testing.assert_array_equal(got[0].cpu().double().numpy(), q)


def swiglu64(h):
    h = h.double().numpy()
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    with np.errstate(over="ignore"):
        return g * 1 / (1 + np.exp(-g)) * u


# exp (2 steps, argument up to 90: 90 more near the ends, where the value is as good as 0 or 1), division 2, products 2
SILU = 2.0 ** -24 * 16


@pytest.mark.parametrize("P,inter", [(1, 128), (33, 256), (70, 2048), (5, 1920)])
def test_swiglu_fp8(P, inter):
    g = gen(P + inter)
    h = normal(g, P, 2 * inter, std=2.0)
    h[0, :2] = torch.tensor([-60.0, 60.0], dtype=torch.bfloat16)
    if P > 3:
        h[2] = 0
        h[3] *= 1e4 ** 0.5
    r = qgg.swiglu_fp8(h.to(DEV), want=("a", "a8", "h8"))
    ref = swiglu64(h)
    gate = np.abs(h[:, :inter].double().numpy())
    slack = (SILU + H32 * gate) * np.abs(ref) + 1e-37
    a = r["a"].cpu().double().numpy()
    assert np.all(np.abs(a - ref) <= HBF * np.abs(ref) + 1.01 * slack)
    check_rows((r["a8"], r["a8_scales"]), ref, slack)
    check_exact((r["a8"], r["a8_scales"]), ref)
    q, s = quantize64(h.double().numpy())
    np.testing.assert_array_equal(r["h8"].cpu().double().numpy(), q)
    np.testing.assert_array_equal(r["h8_scales"].cpu().double().numpy(), s)
    # each output alone is the same
    for name in ("a", "a8", "h8"):
        one = qgg.swiglu_fp8(h.to(DEV), want=(name,))
        assert torch.equal(one[name].view(torch.uint8), r[name].view(torch.uint8))


def test_swiglu_codes_of_many_rows():
    """4 million values, far and near: fp32 arithmetic alone would get some tens of codes wrong."""
    h = normal(gen(99), 1024, 8192, std=3.0)
    h[::7] *= 8
    h[5::31, ::3] = -100
    r = qgg.swiglu_fp8(h.to(DEV), want=("a8",))
    check_exact((r["a8"], r["a8_scales"]), swiglu64(h))


def test_swiglu_values_that_are_not_finite():
    h = normal(gen(6), 4, 512)
    h[0, 3], h[1, 300], h[2, 5], h[3, 7] = float("nan"), float("inf"), float("-inf"), float("inf")
    r = qgg.swiglu_fp8(h.to(DEV))
    fine = normal(gen(6), 4, 512)
    want = torch.from_numpy(swiglu64(fine))
    for i, c in ((0, 3), (1, 44), (2, 5), (3, 7)):
        assert torch.isnan(r["a8"][i, c].float())
        want[i, c] = float("nan")
    check_exact((r["a8"], r["a8_scales"]), want.numpy())


def perm_of(ids, E):
    p, _ = qgg.expert_permute(ids.to(DEV), E)
    return p


def swiglu_bwd64(da, h, gates, perm, live):
    h, da = np.asarray(h, np.float64), da.double().numpy()
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    f = 1 / (1 + np.exp(-g))
    gp = np.zeros(len(h))
    gp[:live] = gates.double().numpy().reshape(-1)[perm[:live]]
    d = da * gp[:, None]
    dgates = np.zeros(gates.numel())
    dgates[perm[:live]] = (da * g * f * u).sum(1)[:live]
    dh = np.concatenate([d * u * f * (1 + g * (1 - f)), d * g * f], 1)
    size = np.concatenate([np.abs(d * u) * (f + np.abs(g) * f * (1 - f)), np.abs(d * g * f)], 1)
    return dh, size, dgates.reshape(gates.shape), np.abs(da * g * f * u)


@pytest.mark.parametrize("T,k,inter", [(1, 1, 128), (13, 3, 256), (37, 8, 2048), (6, 2, 1920)])
@pytest.mark.parametrize("drop", [False, True])
def test_swiglu_fp8_bwd(T, k, inter, drop):
    E = max(2 * k, 4)
    g = gen(T * 100 + inter)
    P = T * k
    ids = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :k].to(torch.int32)
    if drop:
        ids[0, 0] = -1
        ids[-1, -1] = E + 3
    p = perm_of(ids, E)
    live = int(p.offsets[-1])
    h8, hs = qgg.fp8_quantize(normal(g, P, 2 * inter, std=2.0).to(DEV))
    da = normal(g, P, inter)
    gates = torch.softmax(normal(g, T, k, dtype=torch.float32), 1)
    r = qgg.swiglu_fp8_bwd(da.to(DEV), h8, hs, gates.to(DEV), p, want=("dh", "dh8", "dgates"))
    h = value(h8, hs)
    dh, size, dgates, terms = swiglu_bwd64(da, h, gates, p.perm.cpu().numpy(), live)
    slack = (SILU + H32 * (np.abs(np.tile(h[:, :inter], 2)) + 8)) * size + 1e-37
    got = r["dh"].cpu().double().numpy()
    assert np.all(np.abs(got - dh)[:live] <= (HBF * np.abs(dh) + 1.01 * slack)[:live])
    check_rows((r["dh8"][:live], r["dh8_scales"][:live]), dh[:live], slack[:live])
    check_exact((r["dh8"][:live], r["dh8_scales"][:live]), dh[:live])
    # a sum of `inter` terms in fp32: a lane adds inter / 32, then 8 levels
    tol = np.zeros(P)
    perm = p.perm.cpu().numpy()[:live]
    tol[perm] = ((SILU + H32 * (inter / 16 + 10 + np.abs(h[:, :inter]))) * terms).sum(1)[:live]
    err = np.abs(r["dgates"].cpu().double().numpy() - dgates).reshape(-1)
    assert np.all(err <= tol + 1e-37)
    if drop:
        assert r["dgates"][0, 0] == 0 and r["dgates"][-1, -1] == 0


@pytest.mark.parametrize("down", [-20, -30, -34, -40, -46])
def test_swiglu_fp8_bwd_of_tiny_gradients(down):
    # gates times da below the normal numbers of 32 bits
    g = gen(40 - down)
    T, k, I = 16, 2, 512
    p = perm_of(torch.tensor([[0, 1]] * T, dtype=torch.int32), 2)
    h = normal(g, T * k, 2 * I, std=2.0)
    h[:, I:] *= 2.0 ** 12
    h8, hs = qgg.fp8_quantize(h.to(DEV))
    da = normal(g, T * k, I) * 2.0 ** down
    gates = (torch.rand(T, k, generator=g) + 0.5) * 2.0 ** -100
    r = qgg.swiglu_fp8_bwd(da.to(DEV), h8, hs, gates.to(DEV), p, want=("dh8",))
    dh = swiglu_bwd64(da, value(h8, hs), gates, p.perm.cpu().numpy(), T * k)[0]
    check_exact((r["dh8"], r["dh8_scales"]), dh)


def test_swiglu_gradient_by_differences():
    g = gen(3)
    T, k, I = 2, 2, 128
    ids = torch.tensor([[0, 1], [1, 2]], dtype=torch.int32)
    p = perm_of(ids, 4)
    h8, hs = qgg.fp8_quantize(normal(g, T * k, 2 * I).to(DEV))
    da, gates = normal(g, T * k, I), torch.rand(T, k, generator=g)
    r = qgg.swiglu_fp8_bwd(da.to(DEV), h8, hs, gates.to(DEV), p, want=("dh", "dgates"))
    h, perm = value(h8, hs), p.perm.cpu().numpy()

    def loss(x, gt):                        # sum over rows of gate <da, swiglu(h)>, 64 bits
        a = x[:, :I] / (1 + np.exp(-x[:, :I])) * x[:, I:]
        return (gt.reshape(-1)[perm] * (da.double().numpy() * a).sum(1)).sum()

    gt = gates.double().numpy()
    rng = np.random.RandomState(0)
    for _ in range(60):
        i, c = rng.randint(T * k), rng.randint(2 * I)
        d = np.zeros_like(h)
        d[i, c] = 1e-4
        diff = (loss(h + d, gt) - loss(h - d, gt)) / 2e-4
        assert abs(diff - r["dh"][i, c].item()) <= 2 * HBF * abs(diff) + 1e-5
    for i in range(T):
        for j in range(k):
            d = np.zeros_like(gt)
            d[i, j] = 1e-3
            diff = (loss(h, gt + d) - loss(h, gt - d)) / 2e-3
            assert abs(diff - r["dgates"][i, j].item()) <= 1e-4


def test_swiglu_leaves_rows_behind_the_last():
    g = gen(8)
    ids = torch.tensor([[0, -1], [2, 9], [1, 0]], dtype=torch.int32)
    p = perm_of(ids, 4)
    live = int(p.offsets[-1])
    assert live == 4
    h = normal(g, 6, 512).to(DEV)
    full = qgg.swiglu_fp8(h, want=("a", "a8", "h8"))
    L, f = qgg.lib(), {n: torch.full_like(t.view(torch.uint8), 0x5A) for n, t in full.items()}
    import ctypes
    off = ctypes.c_void_p(p.offsets.data_ptr() + 16)
    assert L.moe_swiglu_fp8(qgg._ptr(h), off, 6, 256, *(qgg._ptr(f[n]) for n in ("a", "a8", "a8_scales", "h8", "h8_scales")),
                            qgg._stream()) == 0
    for n, t in f.items():
        assert torch.equal(t[:live], full[n].view(torch.uint8)[:live]) and torch.all(t[live:] == 0x5A)
    gates = torch.ones(3, 2, device=DEV)
    b = {n: torch.full((6, w), 0x5A, dtype=torch.uint8, device=DEV) for n, w in (("dh", 1024), ("dh8", 512), ("dh8_scales", 4))}
    pc = p.c()
    da = normal(g, 6, 256).to(DEV)
    assert L.moe_swiglu_fp8_bwd(qgg._ptr(da), qgg._ptr(full["h8"]), qgg._ptr(full["h8_scales"]), qgg._ptr(gates),
                                ctypes.byref(pc), 3, 2, 256, qgg._ptr(b["dh"]), qgg._ptr(b["dh8"]),
                                qgg._ptr(b["dh8_scales"]), None, qgg._stream()) == 0
    for t in b.values():
        assert torch.all(t[live:] == 0x5A)


# ------------------------------------------------------------------ grouped product

def weights(g, E, N, K, f32):
    codes = normal(g, E, N, K, std=60.0, dtype=torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn)
    shape = (E, -(-N // 128), K // 128)
    if f32:
        scales = torch.rand(shape, generator=g) * 0.01 + 1e-4
    else:
        scales = torch.randint(112, 124, shape, generator=g).to(torch.uint8).view(torch.float8_e8m0fnu)
    return qgg.Fp8Weight(codes.to(DEV), scales.to(DEV))


def weight_value(w, e):
    s = w.scales[e].cpu().double().repeat_interleave(128, 0)[:w.N].repeat_interleave(128, 1)
    return w.codes[e].cpu().double() * s


# What one 16x16x128 FP8 matrix instruction does to its products, read from one-product and two-product inputs on an
# MI355X: eight consecutive reduced values form a group; a group's products are aligned to its largest exponent sum E and
# cut towards zero below 2^(E - 13) (1 + 2^-13 is kept, 1 + 2^-14 is not, at every E tried and with either sign; a product in
# the next group keeps its bits).  The largest product is at least 2^E and loses nothing (its 8 bits fit), each of the
# other seven loses less than 2^(E - 13): a group is off by less than 7 * 2^-13 times its largest product.  Group sums
# and the accumulator are added in fp32, cut or rounded: at most one step, 2 H32, of what is added so far each.
CUT = 7 * 2.0 ** -13


def largest_products(x, m):
    """sum over the groups of eight reduced values of max |x_r m_rc|, [rows, columns]."""
    x, m = x.abs().float(), m.abs().float()
    total = torch.zeros(x.shape[0], m.shape[1])
    for r in range(0, x.shape[1], 8):
        total += (x[:, r:r + 8, None] * m[None, r:r + 8]).amax(1)
    return total.double()


def check_gemm(w, rows, p, T, k, flags, y):
    """Every element: BF16's rounding, the matrix core's cut, and fp32 additions of the group sums."""
    a = torch.from_numpy(value(*rows))
    trans = bool(flags & qgg.TRANSPOSE_W)
    off, perm = p.offsets.cpu().tolist(), p.perm.cpu().long()
    y = y.cpu().double()
    for e in range(w.E):
        i = torch.arange(off[e], off[e + 1])
        if not len(i):
            continue
        x = a[perm[i] // k] if flags & qgg.A_TOKENS else a[i]
        m = weight_value(w, e)
        m = m if trans else m.t()
        ref = x @ m
        tol = 1.01 * (HBF * ref.abs() + CUT * largest_products(x, m) + (x.shape[1] / 8 + 2) * 2 * H32 * (x.abs() @ m.abs()))
        err = (y[i] - ref).abs()
        assert torch.all(err <= tol), (e, len(i), (err / tol).max())


GEMM = [
    dict(T=1, E=4, k=1, N=64, K=128), dict(T=1, E=8, k=8, N=192, K=256), dict(T=5, E=3, k=2, N=320, K=384),
    dict(T=33, E=4, k=2, N=256, K=512), dict(T=64, E=2, k=1, N=512, K=128), dict(T=130, E=3, k=2, N=448, K=640),
    dict(T=200, E=1, k=1, N=128, K=256), dict(T=300, E=9, k=3, N=64, K=1024), dict(T=70, E=40, k=8, N=576, K=256),
    dict(T=257, E=2, k=2, N=704, K=1152),
]


@pytest.mark.parametrize("f32", [False, True], ids=["e8m0", "fp32"])
@pytest.mark.parametrize("trans", [False, True], ids=["nt", "t"])
@pytest.mark.parametrize("c", GEMM, ids=lambda c: "T{T}E{E}k{k}N{N}K{K}".format(**c))
def test_fp8_grouped_gemm(c, trans, f32):
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    g = gen(T * E + N)
    w = weights(g, E, N, K, f32)
    skew = torch.rand(T, E, generator=g) + torch.arange(E) * 0.1
    p = perm_of(torch.argsort(skew, dim=1, descending=True)[:, :k].to(torch.int32), E)
    for flags in (qgg.A_TOKENS, qgg.A_SORTED):
        x = normal(g, T if flags else T * k, N if trans else K)
        x[0] *= 1e-3
        rows = qgg.fp8_quantize(x.to(DEV))
        f = flags | (qgg.TRANSPOSE_W if trans else 0)
        y = qgg.fp8_grouped_gemm(w, *rows, p, T, k, flags=f)
        check_gemm(w, rows, p, T, k, f, y)
        again = qgg.fp8_grouped_gemm(w, *rows, p, T, k, flags=f)
        assert torch.equal(again, y)


# one expert whose rows fill a tile of 288 to each of its heights, and the first that need two tiles; more than 64
# blocks of reduced columns, so that the scales are staged twice
@pytest.mark.parametrize("rows", [65, 97, 150, 190, 256, 257, 288, 289, 577])
@pytest.mark.parametrize("trans", [False, True], ids=["nt", "t"])
def test_fp8_grouped_gemm_tile_heights(rows, trans):
    g = gen(rows)
    N, K = (8384, 128) if trans else (128, 8448)
    w = weights(g, 1, N, K, rows % 2 == 0)
    p = perm_of(torch.zeros((rows, 1), dtype=torch.int32), 1)
    x = qgg.fp8_quantize(normal(g, rows, N if trans else K).to(DEV))
    flags = qgg.A_TOKENS | (qgg.TRANSPOSE_W if trans else 0)
    check_gemm(w, x, p, rows, 1, flags, qgg.fp8_grouped_gemm(w, *x, p, rows, 1, flags=flags))


def test_fp8_grouped_gemm_one_hot_reads_every_weight():
    # rows that are unit vectors read W back exactly, in both directions
    g = gen(77)
    E, N, K = 2, 320, 256
    w = weights(g, E, N, K, False)
    for trans in (False, True):
        n = N if trans else K
        x = torch.cat([torch.eye(n), torch.eye(n)]).to(torch.bfloat16).to(DEV)
        ids = torch.cat([torch.zeros(n), torch.ones(n)]).to(torch.int32).view(-1, 1)
        p = perm_of(ids, E)
        y = qgg.fp8_grouped_gemm(w, *qgg.fp8_quantize(x), p, 2 * n, 1, flags=qgg.A_TOKENS | (qgg.TRANSPOSE_W if trans else 0))
        for e in range(E):
            want = weight_value(w, e)
            want = want if trans else want.t()
            assert torch.equal(y[e * n:(e + 1) * n].cpu().double(), want.to(torch.bfloat16).double())


@pytest.mark.parametrize("trans", [False, True], ids=["nt", "t"])
def test_fp8_grouped_gemm_dropped_pairs_and_nan(trans):
    g = gen(21)
    T, E, k, N, K = 40, 6, 2, 192, 256
    w = weights(g, E, N, K, False)
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    ids[3, 0], ids[9, 1], ids[39, 1] = -1, E, 1000
    p = perm_of(ids, E)
    live = int(p.offsets[-1])
    assert live == T * k - 3
    x = normal(g, T, N if trans else K)
    x[5, 7] = float("nan")
    rows = qgg.fp8_quantize(x.to(DEV))
    out = torch.full((T * k, K if trans else N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = qgg.fp8_grouped_gemm(w, *rows, p, T, k, flags=qgg.A_TOKENS | (qgg.TRANSPOSE_W if trans else 0), out=out)
    assert y is out and torch.all(y[live:] == 7.0)
    token = p.perm[:live] // k
    nan = torch.isnan(y[:live]).all(1)
    assert torch.equal(nan, token == 5)
    assert torch.isfinite(y[:live][~nan]).all()


def test_fp8_grouped_gemm_long_rows():
    # the widest reduction the call takes, both ways
    g = gen(4)
    T, E, k = 20, 2, 1
    for trans, N, K in ((False, 64, 32768), (True, 32768, 128)):
        w = weights(g, E, N, K, trans)
        p = perm_of((torch.arange(T) % E).to(torch.int32).view(-1, 1), E)
        rows = qgg.fp8_quantize(normal(g, T, 32768).to(DEV))
        f = qgg.A_TOKENS | (qgg.TRANSPOSE_W if trans else 0)
        check_gemm(w, rows, p, T, k, f, qgg.fp8_grouped_gemm(w, *rows, p, T, k, flags=f))


def test_fp8_grouped_gemm_millions_of_rows_of_one_expert():
    # the tiles' shares of the row blocks pass 32 bits
    T, N, K = 4_000_003, 64, 128
    g = gen(77)
    w = weights(g, 1, N, K, False)
    p = perm_of(torch.zeros((T, 1), dtype=torch.int32), 1)
    few = normal(g, 4099, K).to(DEV)
    codes, scales = qgg.fp8_quantize(few)
    source = torch.arange(T, device=DEV) % len(few)
    a = codes.view(torch.uint8)[source].contiguous()
    y = qgg.fp8_grouped_gemm(w, a, scales.view(torch.uint8)[source].contiguous(), p, T, 1)
    small = perm_of(torch.zeros((len(few), 1), dtype=torch.int32), 1)
    one = qgg.fp8_grouped_gemm(w, codes, scales, small, len(few), 1)
    check_gemm(w, (codes, scales), small, len(few), 1, qgg.A_TOKENS, one)
    # a row's result does not hang on the rows beside it
    assert torch.equal(y, one[source[p.perm.long()]])


def test_empty_batches():
    g = gen(1)
    w = weights(g, 4, 128, 256, False)
    p = perm_of(torch.empty((0, 2), dtype=torch.int32), 4)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    rows = qgg.fp8_quantize(x)
    assert qgg.fp8_dequantize(*rows).shape == (0, 256)
    p.perm = p.inv_perm = torch.empty(1, dtype=torch.int32, device=DEV)
    assert qgg.fp8_grouped_gemm(w, *rows, p, 0, 2).shape == (0, 128)
    assert qgg.swiglu_fp8(x)["a8"].shape == (0, 128)
    r = qgg.swiglu_fp8_bwd(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV), *rows, torch.empty((0, 2), device=DEV), p)
    assert r["dgates"].shape == (0, 2)
    ids, _ = qgg.moe_route_scored(torch.empty((0, 8), device=DEV), 2)
    assert ids.shape == (0, 2)
    assert qgg.moe_route_scored_bwd(torch.empty((0, 8), device=DEV), ids, torch.empty((0, 2), device=DEV)).shape == (0, 8)
    assert qgg.moe_combine(x, p, 0, 2).shape == (0, 256)


# ------------------------------------------------------------------ together

def layer(x, logits, bias, w_gu, w_dn, dy, k):
    """One FP8 expert layer, forward and backward, as a training step runs it."""
    T = x.shape[0]
    route = dict(score="sigmoid", renorm=True, scale=2.5)
    ids, gates = qgg.moe_route_scored(logits, k, bias=bias, n_group=4, topk_group=2, **route)
    p, _ = qgg.expert_permute(ids, w_gu.E)
    x8 = qgg.fp8_quantize(x)
    h = qgg.fp8_grouped_gemm(w_gu, *x8, p, T, k)
    s = qgg.swiglu_fp8(h, perm=p)
    o = qgg.fp8_grouped_gemm(w_dn, s["a8"], s["a8_scales"], p, T, k, flags=qgg.A_SORTED)
    y = qgg.moe_combine(o, p, T, k, gates)
    da = qgg.fp8_grouped_gemm(w_dn, *qgg.fp8_quantize(dy), p, T, k, flags=qgg.A_TOKENS | qgg.TRANSPOSE_W)
    b = qgg.swiglu_fp8_bwd(da, s["h8"], s["h8_scales"], gates, p)
    dxp = qgg.fp8_grouped_gemm(w_gu, b["dh8"], b["dh8_scales"], p, T, k, flags=qgg.A_SORTED | qgg.TRANSPOSE_W)
    dx = qgg.moe_combine(dxp, p, T, k)
    dl = qgg.moe_route_scored_bwd(logits, ids, b["dgates"], **route)
    return dict(ids=ids, gates=gates, y=y, dx=dx, dl=dl)


def layer_inputs(seed=31, T=75, E=16, k=4, d=512, inter=256):
    g = gen(seed)
    w_gu, w_dn = weights(g, E, 2 * inter, d, False), weights(g, E, d, inter, True)
    x, dy = normal(g, T, d, std=0.1).to(DEV), normal(g, T, d).to(DEV)
    logits = normal(g, T, E, dtype=torch.float32).to(DEV)
    return x, logits, normal(g, E, std=0.05, dtype=torch.float32).to(DEV), w_gu, w_dn, dy, k


def test_layer_together():
    a = layer_inputs()
    x, logits, bias, w_gu, w_dn, dy, k = a
    r = layer(*a)
    T, d = x.shape
    ids = r["ids"].cpu().long()
    # 64-bit autograd of the layer without any 8-bit rounding of its rows
    xs = x.cpu().double().requires_grad_()
    ls = logits.cpu().double().requires_grad_()
    s = torch.gather(torch.special.expit(ls), 1, ids)
    gates = 2.5 * s / s.sum(1, keepdim=True)
    W1 = torch.stack([weight_value(w_gu, e) for e in range(w_gu.E)])
    W2 = torch.stack([weight_value(w_dn, e) for e in range(w_dn.E)])
    y = 0
    for j in range(k):
        h = torch.bmm(W1[ids[:, j]], xs[:, :, None])[:, :, 0]
        I = h.shape[1] // 2
        o = torch.bmm(W2[ids[:, j]], (torch.nn.functional.silu(h[:, :I]) * h[:, I:])[:, :, None])[:, :, 0]
        y = y + gates[:, j:j + 1] * o
    (y * dy.cpu().double()).sum().backward()
    far = lambda u, v: float((u.detach().cpu().double() - v.detach()).norm() / v.detach().norm())  # noqa: E731
    # a rounding to E4M3 is uniform within half a step: 2^-4 / sqrt 3 = 3.6 % of a value at most, rms.  y passes two
    # (x, a), the second on values that carry the first through a product of two factors (x sqrt 2); dx four (dy, h twice
    # through u and silu', dh); dgates the same with dy and h.  Root of the sums of squares, and a margin of 1.5:
    assert far(r["y"], y) <= 1.5 * 0.036 * (1 + 2) ** 0.5
    assert far(r["dx"], xs.grad) <= 1.5 * 0.036 * (1 + 2 + 2 + 2 + 1) ** 0.5
    assert far(r["dl"], ls.grad) <= 1.5 * 0.036 * (1 + 2 + 2 + 2) ** 0.5


def test_layer_in_graphs_and_streams():
    """Two captured layers replayed in turn with eager work between, and a layer on a side stream."""
    first, second = layer_inputs(31), layer_inputs(47, T=20)
    want = [layer(*first), layer(*second)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer(*first)
    torch.cuda.synchronize()
    for n in other:
        assert torch.equal(other[n], want[0][n]), n
    graphs, outs = [], []
    for a in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(*a))
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
        eager = layer(*second)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for n in w:
                assert torch.equal(o[n], w[n]), n
        for n in eager:
            assert torch.equal(eager[n], want[1][n]), n
        for o in outs:
            for t in o.values():
                t.zero_()


@pytest.mark.parametrize("fmt", [qgg.FMT_MXFP4, qgg.FMT_INT4])
def test_checkpoint_in_the_4bit_backward(fmt):
    """The 4-bit FFN's backward from the 8-bit checkpoint: moe_router_bwd on its values, and the chain of products
    around swiglu_fp8_bwd, agree."""
    import synth.configs as sc

    from .gpu_util import dev_bf16, dev_weights
    cfg = sc.scaled(sc.CONFIGS["mxfp4_ffn_prefill"], T=90, d=512, E=8, k=2, N=512, inter=256, fmt=fmt)
    w_gu, w_dn = (qgg.repack(dev_weights(fmt, *w)) for w in (sc.first_weights(cfg), sc.down_weights(cfg)))
    x, dy = dev_bf16(sc.activations(cfg)), dev_bf16(sc.grad_output(cfg))
    T, k = cfg.T, cfg.k
    f = qgg.moe_ffn_fwd(w_gu, w_dn, x, torch.from_numpy(sc.router_logits(cfg)).to(DEV), k, save_h=True)
    s = qgg.swiglu_fp8(f["h"], perm=f["perm"], want=("a", "h8"))
    # the output recomputed from h, through the down projection and the combine, is the forward's
    o = qgg.dequant_grouped_gemm(w_dn, s["a"], f["perm"], T, k, flags=qgg.A_SORTED)
    y = qgg.moe_combine(o, f["perm"], T, k, f["topk_gates"])
    # h is rounded to BF16 before a here and not there: each of a's two factors by 2^-8, a, o, y by 2^-8 each, rms / sqrt 3
    assert (y.float() - f["y"].float()).norm() <= 3 * HBF * f["y"].float().norm()
    hq = qgg.fp8_dequantize(s["h8"], s["h8_scales"])
    want = qgg.moe_router_bwd(w_gu, w_dn, dy, f["topk_ids"], f["topk_gates"], f["perm"], hq, k)
    da = qgg.dequant_grouped_gemm(w_dn, dy, f["perm"], T, k, flags=qgg.A_TOKENS | qgg.TRANSPOSE_W)
    b = qgg.swiglu_fp8_bwd(da, s["h8"], s["h8_scales"], f["topk_gates"], f["perm"], want=("dh", "dgates"))
    dxp = qgg.dequant_grouped_gemm(w_gu, b["dh"], f["perm"], T, k, flags=qgg.A_SORTED | qgg.TRANSPOSE_W)
    dx = qgg.moe_combine(dxp, f["perm"], T, k)
    assert (dx.float() - want["dx"].float()).norm() <= 3 * HBF * want["dx"].float().norm()
    assert (b["dgates"] - want["dgates"]).norm() <= 3 * HBF * want["dgates"].norm()
