"""Routing to experts and the experts' products against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import fp4
from test_gpu_fp4_gemm import check as check_mm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq

FMTS = ["nvfp4", "mxfp4"]


# ---------------------------------------------------------------- router
def check_route(l, k, **kw):
    """ids equal; weights to fp32: exp, a sum of up to 512 terms in a tree and two divisions, each
    good to a few ulp: 2^-24 (2 + log2 512 + 2 ulp expf twice + ...) < 2^-19."""
    w, ids = fq.fp8q_moe_route(l, k, **kw)
    host = {"groups": kw.get("num_groups", 1), "topg": kw.get("topk_groups", 1), "renorm": kw.get("renormalize", True),
            "scale": float(np.float32(kw.get("scale", 1.0)))}
    bias = kw.get("bias")
    ww, wi = fp4.route(l.double().cpu().numpy(), k, kw.get("scoring", "softmax"),
                       None if bias is None else bias.double().cpu().numpy(), **host)
    np.testing.assert_array_equal(ids.cpu().numpy(), wi)
    np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=2.0 ** -19, atol=1e-37)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,tg", [(1, 8, 2, 1, 1), (1, 128, 8, 1, 1), (7, 33, 5, 1, 1), (65, 64, 8, 8, 3),
                                        (300, 256, 8, 8, 4), (9, 512, 32, 16, 2), (100, 60, 6, 4, 2), (5, 1, 1, 1, 1),
                                        (40, 32, 4, 32, 9), (8, 160, 6, 8, 3)])
def test_route(scoring, T, E, k, G, tg):
    g = torch.Generator(device="cuda").manual_seed(T * E)
    for dtype in (torch.float32, torch.bfloat16):
        l = (2 * torch.randn(T, E + 3, device="cuda", generator=g)).to(dtype)[:, :E]     # wider rows
        for bias in (None, 0.3 * torch.randn(E, device="cuda", generator=g)):
            for renorm in (True, False):
                check_route(l, k, scoring=scoring, bias=bias, num_groups=G, topk_groups=tg, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_and_masks(scoring, biased):
    E = 40
    l = torch.zeros(12, E, device="cuda")
    l[1, 7] = -0.0
    l[2] = torch.arange(E, device="cuda") % 3
    l[3, 5:] = float("-inf")
    l[4] = float("-inf")
    l[5, 3] = float("inf")
    l[6, 3] = l[6, 30] = float("inf")
    l[7] = float("nan")
    l[7, 9] = 1
    l[8] = torch.finfo(torch.float32).min
    l[9] = -1e4
    l[9, 20] = 1e4
    l[10, ::2] = float("-inf")
    l[11] = 80.0
    bias = (torch.arange(E, device="cuda") % 2).float() if biased else None
    for dtype in (torch.float32, torch.bfloat16):
        for kw in (dict(), dict(renormalize=False), dict(num_groups=8, topk_groups=2)):
            check_route(l.to(dtype), 8, scoring=scoring, bias=bias, **kw)


def test_route_near_ties_with_a_bias():
    """Biased keys that differ by a few units of fp32's last place are still ordered."""
    E = 64
    l = torch.linspace(-1, 1, E, device="cuda").repeat(200, 1)
    bias = (0.5 - torch.sigmoid(l[0].double())).float()                # keys of about 0.5, apart by roundings
    check_route(l, 8, scoring="sigmoid", bias=bias)
    check_route(l, 8, scoring="sigmoid", bias=bias, num_groups=8, topk_groups=4)
    check_route(l, 8, scoring="sigmoid", bias=torch.zeros(E, device="cuda"))


def test_route_groups_of_cancelling_biases():
    """A group's two keys of +-4096 sum to little, with the roundings of 4096."""
    E, T = 32, 400
    g = torch.Generator(device="cuda").manual_seed(9)
    l = torch.randn(T, E, device="cuda", generator=g)
    bias = torch.zeros(E, device="cuda")
    bias[0::4], bias[1::4], bias[2::4], bias[3::4] = 4096.0, -4096.0, -5000.0, -5000.0
    check_route(l, 4, scoring="sigmoid", bias=bias, num_groups=8, topk_groups=4)
    check_route(l, 4, scoring="softmax", bias=bias, num_groups=8, topk_groups=4)


@pytest.mark.parametrize("E,G", [(48, 8), (96, 4), (256, 16), (512, 32), (240, 5)])
def test_route_ties_between_groups(E, G):
    """Equal groups and experts: the lowest first, whatever lanes hold them."""
    g = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randint(-2, 3, (200, E), device="cuda", generator=g).float()
    for bias in (None, torch.zeros(E, device="cuda")):
        for scoring in ("softmax", "sigmoid"):
            check_route(l, 6, scoring=scoring, bias=bias, num_groups=G, topk_groups=max(2, G // 3))


def test_route_empty_and_refused():
    w, ids = fq.fp8q_moe_route(torch.zeros(0, 16, device="cuda"), 4)
    assert w.shape == ids.shape == (0, 4)
    l = torch.zeros(2, 16, device="cuda")
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_route(l, 17)
    with pytest.raises(ValueError):
        fq.fp8q_moe_route(l, 2, "tanh")
    with pytest.raises(TypeError):
        fq.fp8q_moe_route(l.half(), 2)
    with pytest.raises(ValueError):
        fq.fp8q_moe_route(l, 2, bias=torch.zeros(15, device="cuda"))


# ---------------------------------------------------------------- plan
@pytest.mark.parametrize("T,k,E", [(1, 8, 128), (1, 1, 1), (333, 6, 64), (512, 8, 8), (513, 8, 512), (4096, 8, 128),
                                   (3000, 5, 33), (20000, 1, 7)])
@pytest.mark.parametrize("kind", ["spread", "one", "absent"])
def test_plan(T, k, E, kind):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "one":
        ids[:] = E // 2                                                # the same expert twice in a token, too
    if kind == "absent":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E
    p = fq.fp8q_moe_plan(torch.from_numpy(ids).cuda(), E)
    for got, want, name in zip(p, fp4.plan(ids, E), p._fields):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
    assert int(p.sf_offsets[-1]) * 128 <= fq.moe_sf_rows(T * k, E)


def test_plan_of_nothing():
    p = fq.fp8q_moe_plan(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 5)
    assert p.offsets.tolist() == p.sf_offsets.tolist() == [0] * 6


# ---------------------------------------------------------------- rows of the experts
def routed(T, k, E, seed, absent=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.choice(E, k, replace=False, p=None) for _ in range(T)]).astype(np.int32)
    ids[:, 0] = np.where(rng.random(T) < 0.5, E - 1, ids[:, 0])        # one crowded expert
    if absent:
        ids[rng.random((T, k)) < absent] = -1
    w = rng.random((T, k)).astype(np.float32)
    return torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()


def weights(E, N, K, fmt, seed):
    """Quantized random weights: (codes [E, N, K/2], blocks, fp64 values [E, N, K])."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, sf, v = [], [], []
    for _ in range(E):
        w = (torch.randn(N, K, device="cuda", generator=g) * 0.05).to(torch.bfloat16)
        a, b = fq.fp8q_fp4_quant(w, fmt)
        q.append(a), sf.append(b), v.append(fq.fp8q_fp4_dequant(a, b, fmt).double())
    return torch.stack(q), torch.stack(sf), torch.stack(v)


def rows_of(plan):
    """Token and expert of each row that exists."""
    pos = plan.pos.cpu().numpy()
    tok = np.full(pos.size, -1)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if pos[t, j] >= 0:
                tok[pos[t, j]] = t
    off = plan.offsets.cpu().numpy()
    exp = np.repeat(np.arange(off.size - 1), np.diff(off))
    return tok[:off[-1]], exp


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,K", [(1, 2, 4, 64), (50, 4, 8, 608), (300, 2, 3, 256)])
def test_scattered_quant(fmt, T, k, E, K):
    ids, _ = routed(T, k, E, 1, 0.2)
    plan = fq.fp8q_moe_plan(ids, E)
    torch.manual_seed(T + K)
    x = torch.randn(T, K + 8, device="cuda").to(torch.bfloat16)[:, :K]
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
    tok, _ = rows_of(plan)
    codes, b = fp4.quantize(x.double().cpu().numpy(), fmt)
    np.testing.assert_array_equal(fp4.unpack(q.cpu().numpy())[:tok.size], codes[tok])
    at = {int(p): int(r) for p, r in zip(plan.pos.flatten(), plan.sf_row.flatten()) if p >= 0}
    got = fp4.load_scales(sf.cpu().numpy(), fq.moe_sf_rows(T * k, E), b.shape[1])
    np.testing.assert_array_equal(got[[at[r] for r in range(tok.size)]], b[tok])


# T chosen so that experts hold none, few, 128, and several tiles of rows; every tile width
CASES = [(1, 2, 4, 128, 64), (20, 2, 8, 272, 160), (130, 2, 2, 400, 256), (600, 3, 5, 528, 96), (2500, 2, 4, 2304, 128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,N,K", CASES)
def test_grouped_mm(fmt, T, k, E, N, K):
    ids, _ = routed(T, k, E, 2, 0.1)
    plan = fq.fp8q_moe_plan(ids, E)
    torch.manual_seed(T + K)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
    w, wsf, wv = weights(E, N, K, fmt, 3)
    y = torch.full((T * k, N), 3.0, dtype=torch.bfloat16, device="cuda")
    gb = torch.rand(E, device="cuda") + 0.5 if fmt == "nvfp4" else None
    fq.fp8q_grouped_mm_fp4(q, w, sf, wsf, fmt, plan, b_gscale=gb, y=y)
    assert fq.fp8q_last_device_status() == fq.OK
    tok, exp = rows_of(plan)
    xv = fq.fp8q_fp4_dequant(*fq.fp8q_fp4_quant(x, fmt), fmt).double()
    for e in range(E):
        at = np.nonzero(exp == e)[0]
        if at.size:
            check_mm(y[at], xv[tok[at]], wv[e], K, 1.0 if gb is None else float(gb[e].double()))
    assert bool((y[tok.size:] == 3).all())                             # rows without an expert stay


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_of_pairs_and_remainders(fmt):
    """Experts of 768 rows and more on average: rows at both sides of 128 and 256, none, and one;
    three calls one after the other."""
    rows = [0, 1, 128, 129, 255, 256, 257, 384, 385, 512, 3 * 256 + 100, 9000]
    E, N, K = len(rows), 272, 544
    ids = torch.cat([torch.full((r,), e, dtype=torch.int32) for e, r in enumerate(rows)] + [torch.full((7,), -1, dtype=torch.int32)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(3))].view(-1, 1).cuda()
    T = len(ids)
    assert T >= 768 * E
    plan = fq.fp8q_moe_plan(ids, E)
    torch.manual_seed(12)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
    w, wsf, wv = weights(E, N, K, fmt, 13)
    y = torch.full((T, N), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        fq.fp8q_grouped_mm_fp4(q, w, sf, wsf, fmt, plan, y=y)
    assert fq.fp8q_last_device_status() == fq.OK
    tok, exp = rows_of(plan)
    xv = fq.fp8q_fp4_dequant(*fq.fp8q_fp4_quant(x, fmt), fmt).double()
    for e in range(E):
        at = np.nonzero(exp == e)[0]
        assert at.size == rows[e]
        if at.size:
            check_mm(y[at], xv[tok[at]], wv[e], K, 1.0)
    assert bool((y[tok.size:] == 3).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,I,K", [(1, 2, 4, 128, 64), (20, 2, 8, 256, 160), (600, 3, 5, 384, 96), (2500, 2, 4, 2304, 128)])
def test_silu_quant_epilogue(fmt, T, k, E, I, K):
    """Codes and scales of the quantized hidden rows.  The kernel's y differs from the definition's
    by its fp32 accumulation and SiLU (below 2^-15 of the largest term; gate and up are sums whose
    own error the absolute products bound), so a code may differ by one step where the exact
    quotient lies that near a rounding border, and a group is skipped where its scale does.  How many
    that may be: the tolerance is about 2^-13 of a typical y, and a scale's borders lie 2^-3 to 2^-4
    apart, a code's 2^-2: about 2e-3 of the groups and values.  They fall independently, so a count of
    mean m stays below m + 5 sqrt(m) + 5 (Poisson, 1e-6)."""
    ids, _ = routed(T, k, E, 4, 0.1)
    plan = fq.fp8q_moe_plan(ids, E)
    torch.manual_seed(T + K)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
    w, wsf, wv = weights(E, 2 * I, K, fmt, 5)
    gh = torch.tensor([0.0113], device="cuda") if fmt == "nvfp4" else None
    hq, hsf = fq.fp8q_grouped_mm_fp4_silu_quant(q, w, sf, wsf, fmt, plan, gscale=gh)
    assert fq.fp8q_last_device_status() == fq.OK
    tok, exp = rows_of(plan)
    xv = fq.fp8q_fp4_dequant(*fq.fp8q_fp4_quant(x, fmt), fmt).double()
    at = {int(p): int(r) for p, r in zip(plan.pos.flatten(), plan.sf_row.flatten()) if p >= 0}
    G = fp4.GROUP[fmt]
    bytes_ = fp4.load_scales(hsf.cpu().numpy(), fq.moe_sf_rows(T * k, E), I // G)[[at[r] for r in range(tok.size)]]
    codes = fp4.unpack(hq.cpu().numpy())[:tok.size]
    g = 1.0 if gh is None else float(gh.double())
    moved = total = skipped = 0
    for e in range(E):
        r = np.nonzero(exp == e)[0]
        if not r.size:
            continue
        h = xv[tok[r]] @ wv[e].t()
        ab = xv[tok[r]].abs() @ wv[e].abs().t()
        tol = ((K / 64) * 2.0 ** -23 + 2.0 ** -18) * ab
        h, tol = h.cpu().numpy(), tol.cpu().numpy()
        y = fp4.silu_mul(h[:, :I], h[:, I:])
        # |d silu| <= 1.1 |d gate|, |silu(g)| <= |g|
        ey = 1.1 * tol[:, :I] * np.abs(h[:, I:]) + np.abs(h[:, :I]) * tol[:, I:] + 2.0 ** -19 * np.abs(y) + 1e-30
        lo, hi = (fp4.quantize(np.copysign(np.maximum(np.abs(y) + s * ey, 0), y), fmt, g) for s in (-1, 1))
        # the group's scale is decided where both ends of its amax agree
        same = lo[1] == hi[1]
        skipped += int((~same).sum())
        np.testing.assert_array_equal(bytes_[r][same], lo[1][same])
        wide = np.repeat(same, G, axis=1)
        got = codes[r]
        ok = (got == lo[0]) | (got == hi[0]) | (np.abs(y) <= ey)
        assert ok[wide].all()
        moved += int((got != fp4.quantize(y, fmt, g)[0])[wide].sum())
        total += int(wide.sum())
    for n, of in ((skipped, total / G), (moved, total)):
        assert n <= 2e-3 * of + 5 * (2e-3 * of) ** 0.5 + 5


@pytest.mark.parametrize("T,k,H", [(1, 8, 64), (37, 6, 136), (1000, 9, 2048), (3, 32, 8)])
def test_combine(T, k, H):
    """A sum of k fp32 products (k 2^-24 of the absolute sum), rounded once to bf16 (2^-8)."""
    ids, w = routed(T, k, max(k, 40), 6, 0.2)
    plan = fq.fp8q_moe_plan(ids, max(k, 40))
    torch.manual_seed(T + H)
    o = torch.randn(T * k, H + 8, device="cuda").to(torch.bfloat16)[:, :H]
    o[int(plan.offsets[-1]):] = float("nan")                           # rows without an expert
    y = fq.fp8q_moe_combine(o, plan, w)
    pos = plan.pos.long()
    part = torch.where((pos >= 0)[:, :, None], o.double()[pos.clamp(min=0)] * w.double()[:, :, None], 0.0)
    ref, ab = part.sum(1), part.abs().sum(1)
    assert bool(((y.double() - ref).abs() <= (2.0 ** -8) * ref.abs() + (k + 1) * 2.0 ** -23 * ab + 1e-38).all())


# ---------------------------------------------------------------- the whole pass
def parts(x, ids, w, w13, s13, w2, s2, fmt, gx, g13, gh, g2):
    plan = fq.fp8q_moe_plan(ids, w13.shape[0])
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt, gscale=gx)
    q, sf = fq.fp8q_grouped_mm_fp4_silu_quant(q, w13, sf, s13, fmt, plan, a_gscale=gx, b_gscale=g13, gscale=gh)
    return fq.fp8q_moe_combine(fq.fp8q_grouped_mm_fp4(q, w2, sf, s2, fmt, plan, a_gscale=gh, b_gscale=g2), plan, w)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I,absent", [(1, 2, 8, 256, 128, 0), (1, 4, 16, 96, 256, 0.5), (60, 4, 8, 544, 384, 0.1),
                                              (700, 2, 6, 512, 256, 0), (3000, 4, 16, 1024, 128, 0.05)])
def test_experts(fmt, T, k, E, H, I, absent):
    """The one call equals its parts bit for bit, and the fp64 definition within what 4-bit
    quantization of the hidden rows leaves open: a code that moves one step changes y by at most
    2^-2 of its term, and few do, so the whole is held in the norm."""
    ids, w = routed(T, k, E, 7, absent)
    torch.manual_seed(T + H)
    x = torch.randn(T, H + 16, device="cuda").to(torch.bfloat16)[:, :H]
    w13, s13, v13 = weights(E, 2 * I, H, fmt, 8)
    w2, s2, v2 = weights(E, H, I, fmt, 9)
    gx = g13 = gh = g2 = None
    if fmt == "nvfp4":
        gx, gh = torch.tensor([0.0213], device="cuda"), torch.tensor([0.0031], device="cuda")
        g13, g2 = torch.rand(E, device="cuda") + 0.5, torch.rand(E, device="cuda") + 0.5
    y = fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt, x_gscale=gx, w13_gscale=g13, h_gscale=gh, w2_gscale=g2)
    assert fq.fp8q_last_device_status() == fq.OK
    assert torch.equal(y, parts(x, ids, w, w13, s13, w2, s2, fmt, gx, g13, gh, g2))
    one = lambda v: 1.0 if v is None else float(v.double())  # noqa: E731
    xc, xb = fp4.quantize(x.double().cpu().numpy(), fmt, one(gx))
    xv = torch.from_numpy(fp4.values(xc, xb, fmt, one(gx))).cuda()
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            h = (xv[t] @ v13[e].t() * (1.0 if g13 is None else g13[e].double())).cpu().numpy()
            hc, hb = fp4.quantize(fp4.silu_mul(h[:, :I], h[:, I:]), fmt, one(gh))
            hv = torch.from_numpy(fp4.values(hc, hb, fmt, one(gh))).cuda()
            ref.index_add_(0, t, hv @ v2[e].t() * (1.0 if g2 is None else g2[e].double()) * w[t, j].double()[:, None])
    err = float((y.double() - ref).norm() / ref.norm())
    # two bf16 roundings (rms 2^-9 / sqrt(3) each, at most 2^-8) and 2e-3 of the codes a step off
    assert err <= 2 * 2.0 ** -8 + 2e-3 ** 0.5 * 2.0 ** -3, err


def test_experts_graph_streams_and_workspace():
    """Captured and replayed on new inputs, in two graphs with workspaces of their own; on another
    stream; with a larger workspace and a padded y."""
    T, k, E, H, I, fmt = 24, 4, 16, 512, 256, "nvfp4"
    w13, s13, _ = weights(E, 2 * I, H, fmt, 10)
    w2, s2, _ = weights(E, H, I, fmt, 11)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    l = torch.randn(T, E, device="cuda")

    def layer(**kw):
        w, ids = fq.fp8q_moe_route(l, k)
        return fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt, **kw)

    layer()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y = layer()
        graphs.append((gr, y))
    for _ in range(3):
        x.copy_(torch.randn(T, H, device="cuda"))
        l.copy_(torch.randn(T, E, device="cuda"))
        want = layer()
        for gr, y in graphs:
            y.zero_()
            gr.replay()
            assert torch.equal(y, want)
    w, ids = fq.fp8q_moe_route(l, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    big = torch.zeros(T, H + 8, dtype=torch.bfloat16, device="cuda")
    ws = fq.make_moe_workspace(T + 100, k, E, H, I, fmt)
    fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt, y=big[:, :H], workspace=ws)
    assert torch.equal(big[:, :H], want) and not bool(big[:, H:].any())
    assert fq.fp8q_moe_experts_fp4(x[:0], ids[:0], w[:0], w13, s13, w2, s2, fmt).shape == (0, H)
    none = fq.fp8q_moe_experts_fp4(x, torch.full_like(ids, -1), w, w13, s13, w2, s2, fmt)
    assert not bool(none.any())
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt, workspace=ws[256:512])
    with pytest.raises(ValueError):
        fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2[:, :, :64].contiguous(), s2, fmt)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_weights_of_small_scores(scoring, dtype):
    """A bias that decides alone selects experts whose scores are far below the largest, and below
    fp32's range: renormalized, their weights are those of fp64.  (The differences of logits near 100
    are rounded at 2^-18: an exponential of them alone would miss the bound.)"""
    T, E = 300, 64
    g = torch.Generator(device="cuda").manual_seed(21)
    l = (40 * torch.randn(T, E, device="cuda", generator=g)).to(dtype)
    l[:100] -= 300
    bias = 5000 * torch.randn(E, device="cuda", generator=g)
    for renorm in (True, False):
        check_route(l, 6, scoring=scoring, bias=bias, renormalize=renorm)
        check_route(l, 6, scoring=scoring, renormalize=renorm)
