"""The 4-bit and experts part of the C ABI: every function include/fp8q_fp4.h
declares is exported and bound, and arguments are refused on the host (no
kernel is launched by these calls, so they run without a GPU)."""
import ctypes

import pytest
import torch

import fp8_quantized_linear_rms_b200 as fq

L = fq.lib
P = 1 << 20          # an aligned address that is never dereferenced
BAD, UNS, OK = fq.ERR_INVALID_ARG, fq.ERR_UNSUPPORTED, fq.OK
EPS = ctypes.c_float(1e-6)
BIG = 1 << 31


def test_every_declared_function_is_exported_and_bound():
    names = fq.header_functions(fq.FP4_HEADER_PATH)
    assert len(names) == 15
    for n in names:
        assert hasattr(fq.lib, n) and callable(getattr(fq, n)), n
    assert not set(names) & set(fq.header_functions())


def quant(x=P, M=4, K=256, ldx=256, fmt=0, g=None, q=P, ldq=128, sf=P):
    return L.fp8q_fp4_quant(x, M, K, ldx, fmt, g, q, ldq, sf, None)


def test_quant_refusals():
    for kw in (dict(x=None), dict(q=None), dict(sf=None), dict(M=-1), dict(K=0), dict(K=48, ldx=48), dict(ldx=248),
               dict(ldx=260), dict(ldq=120), dict(ldq=132), dict(fmt=2), dict(fmt=-1), dict(fmt=1, g=P), dict(x=P + 8),
               dict(q=P + 8), dict(sf=P + 4), dict(g=P + 2), dict(M=BIG), dict(K=BIG, ldx=BIG, ldq=BIG)):
        assert quant(**kw) == BAD, kw
    assert quant(x=None, q=None, sf=None, M=0) == OK
    assert quant(M=0, K=40) == BAD
    s = L.fp8q_silu_mul_fp4_quant
    assert s(P, 4, 256, 256, 0, None, P, 128, P, None) == BAD          # ldx < 2 I
    assert s(None, 0, 256, 512, 0, None, None, 128, None, None) == OK
    r = L.fp8q_rmsnorm_fp4_quant
    assert r(P, None, EPS, 4, 256, 256, 0, None, P, 128, P, None) == BAD
    assert r(P, P + 2, EPS, 4, 256, 256, 0, None, P, 128, P, None) == BAD
    for eps in (-1.0, float("nan"), float("inf")):
        assert r(P, P, ctypes.c_float(eps), 4, 256, 256, 0, None, P, 128, P, None) == BAD
    assert r(None, None, EPS, 0, 256, 256, 1, None, None, 128, None, None) == OK
    d = L.fp8q_fp4_dequant
    assert d(P, 128, P, 0, None, 4, 256, None, 256, None) == BAD
    assert d(P, 128, P, 0, None, 4, 256, P, 248, None) == BAD
    assert d(P, 120, P, 0, None, 4, 256, P, 256, None) == BAD
    assert d(P, 128, P, 1, P, 4, 256, P, 256, None) == BAD
    assert d(None, 128, None, 1, None, 0, 256, None, 256, None) == OK


def test_scale_bytes():
    assert fq.fp8q_fp4_sf_bytes(1, 32, "nvfp4") == 512
    assert fq.fp8q_fp4_sf_bytes(129, 64 * 3 + 32, "nvfp4") == 2 * 4 * 512
    assert fq.fp8q_fp4_sf_bytes(129, 128 * 3 + 32, "mxfp4") == 2 * 4 * 512
    assert fq.fp4_sf_shape(129, 416, "mxfp4") == (2, 4, 512)
    assert L.fp8q_fp4_sf_bytes(0, 32, 0) == 0 and L.fp8q_fp4_sf_bytes(4, 32, 7) == 0
    with pytest.raises(ValueError):
        fq.fp4_sf_shape(1, 32, "fp4")


def mm(a=P, b=P, asf=P, bsf=P, fmt=0, ga=None, gb=None, M=4, N=64, K=256, y=P, ldy=64):
    return L.fp8q_scaled_mm_fp4(a, b, asf, bsf, fmt, ga, gb, M, N, K, y, ldy, None)


def test_mm_refusals():
    for kw in (dict(a=None), dict(b=None), dict(asf=None), dict(bsf=None), dict(y=None), dict(N=24, ldy=24), dict(N=0),
               dict(K=48), dict(K=0), dict(M=-1), dict(ldy=56), dict(ldy=68), dict(fmt=2), dict(fmt=1, ga=P),
               dict(fmt=1, gb=P), dict(a=P + 8), dict(b=P + 8), dict(asf=P + 8), dict(bsf=P + 8), dict(y=P + 8),
               dict(ga=P + 1), dict(gb=P + 2), dict(M=BIG), dict(N=BIG, ldy=BIG), dict(K=BIG),
               dict(M=1 << 30, N=1 << 30, ldy=1 << 30)):
        assert mm(**kw) == BAD, kw
    assert mm(a=None, b=None, asf=None, bsf=None, y=None, M=0) == OK


def route(l=P, bf=0, T=4, E=64, ld=64, k=8, sc=0, bias=None, G=1, tg=1, rn=1, w=P, ids=P):
    return L.fp8q_moe_route(l, bf, T, E, ld, k, sc, bias, G, tg, rn, ctypes.c_float(1.0), w, ids, None)


def test_route_refusals():
    for kw in (dict(l=None), dict(w=None), dict(ids=None), dict(bf=2), dict(T=-1), dict(E=0), dict(ld=63), dict(k=0),
               dict(sc=2), dict(G=0), dict(tg=0), dict(G=3, tg=1), dict(G=4, tg=5), dict(G=16, tg=1, k=8), dict(k=32, E=16, ld=16),
               dict(rn=2), dict(l=P + 2), dict(bias=P + 2), dict(w=P + 1), dict(ids=P + 1), dict(T=BIG)):
        assert route(**kw) == BAD, kw
    for kw in (dict(E=513, ld=513), dict(k=33), dict(E=64, G=64, tg=64)):
        assert route(**kw) == UNS, kw
    assert route(l=None, w=None, ids=None, T=0) == OK


def test_plan_and_combine_refusals():
    pl = L.fp8q_moe_plan
    assert pl(P, 8, 0, P, P, P, P, None, 0, None) == BAD
    assert pl(P, 8, 513, P, P, P, P, None, 0, None) == UNS
    for i in (0, 3, 4, 5, 6):
        a = [P, 8, 4, P, P, P, P, None, 0, None]
        a[i] = None
        assert pl(*a) == BAD, i
    assert pl(P, -1, 4, P, P, P, P, None, 0, None) == BAD
    n = fq.fp8q_moe_plan_workspace_bytes(65536, 256)
    assert n == 16 * 256 * 4 and fq.fp8q_moe_plan_workspace_bytes(4096, 256) == 0
    assert pl(P, 65536, 256, P, P, P, P, None, 0, None) == BAD
    assert pl(P, 65536, 256, P, P, P, P, P, n - 1, None) == BAD
    c = L.fp8q_moe_combine
    assert c(P, 64, P, P, 4, 2, 60, P, 64, None) == BAD          # H not a multiple of 8
    assert c(P, 56, P, P, 4, 2, 64, P, 64, None) == BAD
    assert c(P, 64, None, P, 4, 2, 64, P, 64, None) == BAD
    assert c(P, 64, P, P, 4, 0, 64, P, 64, None) == BAD
    assert c(None, 64, None, None, 0, 2, 64, None, 64, None) == OK
    q = L.fp8q_moe_fp4_quant
    assert q(P, 4, 256, 256, 0, P, P, 0, None, P, 128, P, None) == BAD
    assert q(P, 4, 256, 256, 2, None, P, 0, None, P, 128, P, None) == BAD
    assert q(None, 0, 256, 256, 2, None, None, 0, None, None, 128, None, None) == OK


def test_grouped_refusals():
    g = L.fp8q_grouped_mm_fp4
    assert g(P, P, P, P, 0, None, None, None, P, 4, 8, 64, 256, P, 64, None) == BAD
    assert g(P, P, P, P, 0, None, None, P, P, 0, 8, 64, 256, P, 64, None) == BAD
    assert g(P, P, P, P, 0, None, None, P, P, 513, 8, 64, 256, P, 64, None) == UNS
    assert g(P, P, P, P, 0, None, None, P, P, 4, 8, 64, 256, P, 56, None) == BAD
    assert g(P, P, P, P, 0, None, None, P, P, 4, 8, 1 << 30, 256, P, 1 << 30, None) == BAD    # E N past 32 bits
    assert g(None, None, None, None, 0, None, None, None, None, 4, 0, 64, 256, None, 64, None) == OK
    s = L.fp8q_grouped_mm_fp4_silu_quant
    assert s(P, P, P, P, 0, None, None, P, P, 4, 8, 192, 256, None, P, P, None) == UNS        # I % 128
    assert s(P, P, P, P, 1, None, None, P, P, 4, 8, 128, 256, P, P, P, None) == BAD           # mxfp4 with gscale
    assert s(P, P, P, P, 0, None, None, P, P, 4, 8, 128, 256, None, None, P, None) == BAD
    assert s(None, None, None, None, 0, None, None, None, None, 4, 0, 128, 256, None, None, None, None) == OK


def experts(**kw):
    a = dict(x=P, T=4, ldx=256, ids=P, w=P, k=2, E=8, H=256, I=128, fmt=0, w13=P, s13=P, w2=P, s2=P, gx=None, g13=None,
             gh=None, g2=None, y=P, ldy=256, ws=P, n=None)
    a.update(kw)
    if a["n"] is None:
        a["n"] = L.fp8q_moe_experts_fp4_workspace_bytes(a["T"], a["k"], a["E"], a["H"], a["I"], a["fmt"])
    return L.fp8q_moe_experts_fp4(*a.values(), None)


def test_experts_refusals():
    n = fq.fp8q_moe_experts_fp4_workspace_bytes(4, 2, 8, 256, 128, "nvfp4")
    assert n > 0 and fq.fp8q_moe_experts_fp4_workspace_bytes(0, 2, 8, 256, 128, "nvfp4") == 0
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(w13=None), dict(s13=None), dict(w2=None), dict(s2=None),
               dict(y=None), dict(ws=None, n=n), dict(n=n - 1), dict(ws=P + 128, n=n), dict(ldx=248), dict(ldy=260),
               dict(H=48, ldx=48, ldy=48), dict(k=0), dict(k=33), dict(E=0), dict(E=513), dict(T=-1), dict(fmt=2),
               dict(fmt=1, gx=P), dict(fmt=1, g2=P), dict(x=P + 8), dict(y=P + 8), dict(w13=P + 8), dict(gh=P + 2),
               dict(T=1 << 30, n=1 << 40)):
        assert experts(**kw) == BAD, kw
    assert experts(I=64, n=n) == UNS
    assert experts(T=0, x=None, ids=None, w=None, w13=None, s13=None, w2=None, s2=None, y=None, ws=None) == OK


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    plan = fq.MoePlan(*(torch.zeros(4, 1, dtype=torch.int32) for _ in range(4)))
    for call in (lambda: fq.fp8q_fp4_quant(x, "nvfp4"), lambda: fq.fp8q_rmsnorm_fp4_quant(x, x[0], 1e-6, "nvfp4"),
                 lambda: fq.fp8q_silu_mul_fp4_quant(x, "mxfp4"), lambda: fq.fp8q_fp4_dequant(u, u, "nvfp4"),
                 lambda: fq.fp8q_scaled_mm_fp4(u, u, u, u, "nvfp4"), lambda: fq.fp8q_moe_route(x, 2),
                 lambda: fq.fp8q_moe_plan(torch.zeros(4, 2, dtype=torch.int32), 8),
                 lambda: fq.fp8q_moe_fp4_quant(x, plan, "nvfp4"),
                 lambda: fq.fp8q_grouped_mm_fp4(u, u[None], u, u, "nvfp4", plan),
                 lambda: fq.fp8q_grouped_mm_fp4_silu_quant(u, u[None], u, u, "nvfp4", plan),
                 lambda: fq.fp8q_moe_combine(x, plan, x),
                 lambda: fq.fp8q_moe_experts_fp4(x, plan.pos, x, u[None], u, u[None], u, "nvfp4")):
        with pytest.raises(TypeError):
            call()


def test_plan_of_more_entries_than_are_ordered():
    big = (1 << 25) + 1
    n = fq.fp8q_moe_plan_workspace_bytes(big, 4)
    assert L.fp8q_moe_plan(P, big, 4, P, P, P, P, P, n, None) == UNS
    assert L.fp8q_moe_plan(P, 1 << 30, 4, P, P, P, P, P, n, None) == BAD
    assert experts(T=big, k=1, n=1 << 50) == BAD
    assert fq.fp8q_moe_experts_fp4_workspace_bytes(big, 1, 8, 256, 128, "nvfp4") == 0
