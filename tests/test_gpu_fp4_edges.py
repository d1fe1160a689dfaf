"""4-bit operators and experts where they can go wrong beside their arithmetic:
offsets past 32 bits, first calls inside a capture, streams side by side, plans
that do not fit, alignments, experts without rows."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq

FMTS = ["nvfp4", "mxfp4"]


def rnd(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32).to(torch.bfloat16)


def experts_weights(E, H, I, fmt, seed):
    w13 = [fq.fp8q_fp4_quant(rnd(2 * I, H, seed=seed + e), fmt) for e in range(E)]
    w2 = [fq.fp8q_fp4_quant(rnd(H, I, seed=seed + 1000 + e), fmt) for e in range(E)]
    return [torch.stack([p[i] for p in w]) for w in (w13, w2) for i in (0, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (16, 0), (16, 8), (8, 8)])
def test_rows_at_any_16_bytes(fmt, pad, shift):
    """Rows and bases at odd multiples of 16 bytes take the 16-byte accesses, with the same results."""
    M, K = 37, 288
    x = rnd(M, K, seed=1)
    q, sf = fq.fp8q_fp4_quant(x, fmt)
    y = fq.fp8q_fp4_dequant(q, sf, fmt)
    room = torch.full(((M + 1) * (K + pad) + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(room, (M, K), (K + pad, 1), shift)
    fq.fp8q_fp4_dequant(q, sf, fmt, y=view)
    assert torch.equal(view, y)
    view.copy_(x)
    q2, sf2 = fq.fp8q_fp4_quant(view, fmt)
    assert torch.equal(q, q2) and torch.equal(fq.fp8q_fp4_dequant(q2, sf2, fmt), y)
    w = rnd(K, seed=2)
    a, b = fq.fp8q_rmsnorm_fp4_quant(x, w, 1e-6, fmt), fq.fp8q_rmsnorm_fp4_quant(view, w, 1e-6, fmt)
    assert torch.equal(a[0], b[0])
    view[:, :] = 7.0
    assert bool((room == 7).all())                                   # nothing was written beside the rows


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """2.2e9 values: the last rows equal those rows alone."""
    M, K = 67500, 32768
    x = rnd(1, K, seed=3).expand(M, K).contiguous()
    tail = rnd(5, K, seed=4)
    x[-5:] = tail
    q, sf = fq.fp8q_fp4_quant(x, fmt)
    del x
    tq, tsf = fq.fp8q_fp4_quant(tail, fmt)
    assert torch.equal(q[-5:], tq)
    y = fq.fp8q_fp4_dequant(q, sf, fmt)
    assert torch.equal(y[-5:], fq.fp8q_fp4_dequant(tq, tsf, fmt))
    del y
    # a product of as many values: rows 0 and the last
    a, asf = q[:, :64].contiguous(), fq.fp8q_fp4_quant(rnd(M, 128, seed=5), fmt)[1]
    b, bsf = fq.fp8q_fp4_quant(rnd(32768, 128, seed=6), fmt)
    del q, sf
    y = fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, fmt)
    assert fq.fp8q_last_device_status() == fq.OK
    first = M // 128 * 128                                           # rows of the last scale block
    part = fq.fp8q_scaled_mm_fp4(a[first:].contiguous(), b, asf[-1:].contiguous(), bsf, fmt)
    assert torch.equal(y[first:], part)


def test_weights_past_32_bits():
    """Experts whose codes take 4.3 GB: the last one's rows equal the dense product with its weights."""
    E, N, K, fmt = 33, 8192, 32768, "nvfp4"
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8, generator=g)
    wsf = torch.randint(0, 100, (E, *fq.fp4_sf_shape(N, K, fmt)), device="cuda", dtype=torch.uint8, generator=g)
    ids = torch.full((200, 1), E - 1, dtype=torch.int32, device="cuda")
    plan = fq.fp8q_moe_plan(ids, E)
    q, sf = fq.fp8q_moe_fp4_quant(rnd(200, K, seed=8), plan, fmt)
    y = fq.fp8q_grouped_mm_fp4(q, w, sf, wsf, fmt, plan)
    assert fq.fp8q_last_device_status() == fq.OK
    dense = fq.fp8q_scaled_mm_fp4(q, w[-1].contiguous(), sf[:2].contiguous(), wsf[-1].contiguous(), fmt)
    # the same products in another order: fp32 accumulation, then a rounding to bf16
    ref = dense.double().abs().clamp(min=float(dense.double().abs().mean()))
    assert bool(((y.double() - dense.double()).abs() <= 2.0 ** -6 * ref).all())


FIRST = r"""
import torch, sys
import fp8_quantized_linear_rms_b200 as fq
T, k, E, H, I, fmt = {T}, 2, 8, 256, 128, "nvfp4"
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
logits = torch.randn(T, E, device="cuda", generator=g)
code = lambda *s: torch.randint(0, 256, s, device="cuda", dtype=torch.uint8, generator=g)
scale = lambda *s: torch.randint(40, 60, s, device="cuda", dtype=torch.uint8, generator=g)
w13, s13 = code(E, 2 * I, H // 2), scale(E, *fq.fp4_sf_shape(2 * I, H, fmt))
w2, s2 = code(E, H, I // 2), scale(E, *fq.fp4_sf_shape(H, I, fmt))
def run():
    w, ids = fq.fp8q_moe_route(logits, k)
    y = fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt)
    q, sf = fq.fp8q_fp4_quant(y, fmt)
    z = fq.fp8q_scaled_mm_fp4(q, w13[0], sf, s13[0], fmt)
    return y, z, fq.fp8q_fp4_dequant(*fq.fp8q_silu_mul_fp4_quant(z, fmt), fmt)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert fq.fp8q_last_device_status() == fq.OK
for a, b in zip(out, run()):
    assert torch.equal(a, b) and bool(a.isfinite().all())
print("same")
"""


@pytest.mark.parametrize("T", [3, 700])
def test_first_calls_inside_a_capture(T):
    r = subprocess.run([sys.executable, "-c", FIRST.format(T=T)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [5, 400])
def test_two_streams_at_once(fmt, T):
    """Passes side by side, each with a workspace of its own, give what they give alone; so do calls
    that take the stream as an argument."""
    k, E, H, I = 4, 16, 512, 256
    w13, s13, w2, s2 = experts_weights(E, H, I, fmt, 20)
    xs, want = [], []
    for s in range(2):
        x = rnd(T, H, seed=30 + s)
        w, ids = fq.fp8q_moe_route(rnd(T, E, seed=40 + s).float(), k)
        xs.append((x, ids, w))
        want.append(fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for s in range(2):
            got[s].append(fq.fp8q_moe_experts_fp4(*xs[s], w13, s13, w2, s2, fmt, stream=streams[s]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[s]) for s in range(2) for y in got[s])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k", [(1, 1), (9, 4), (150, 2)])
def test_no_expert_here(fmt, T, k):
    """Every expert on another GPU (ids of -1, and beyond the last): all zeros."""
    E, H, I = 4, 256, 128
    w13, s13, w2, s2 = experts_weights(E, H, I, fmt, 50)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    ids[:, k // 2:] = E
    y = torch.full((T, H), 5.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8q_moe_experts_fp4(rnd(T, H), ids, torch.ones(T, k, device="cuda"), w13, s13, w2, s2, fmt, y=y)
    assert fq.fp8q_last_device_status() == fq.OK and not bool(y.any())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [126, 128, 129, 132])
def test_both_sides_of_the_small_plan(fmt, n):
    """The pass with and without the one-launch plan: the parts, called one by one, never take it."""
    k, E, H, I = 2, 512, 256, 128
    w13, s13, w2, s2 = (t.expand(E, *t.shape[1:]).contiguous() for t in experts_weights(1, H, I, fmt, 60))
    k = 1 if n % 2 else 2
    T = n // k
    g = torch.Generator(device="cuda").manual_seed(n)
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32, generator=g)
    ids[:3] = E - 1
    ids[-1] = 0
    x, w = rnd(T, H, seed=n), torch.rand(T, k, device="cuda", generator=g)
    y = fq.fp8q_moe_experts_fp4(x, ids, w, w13, s13, w2, s2, fmt)
    plan = fq.fp8q_moe_plan(ids, E)
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
    q, sf = fq.fp8q_grouped_mm_fp4_silu_quant(q, w13, sf, s13, fmt, plan)
    assert torch.equal(y, fq.fp8q_moe_combine(fq.fp8q_grouped_mm_fp4(q, w2, sf, s2, fmt, plan), plan, w))


def test_a_plan_that_does_not_fit():
    """Offsets of another plan, larger than the rows: rows from M on are left alone."""
    E, N, K, M, fmt = 4, 144, 128, 150, "nvfp4"
    w = [fq.fp8q_fp4_quant(rnd(N, K, seed=70 + e), fmt) for e in range(E)]
    b, bsf = torch.stack([v[0] for v in w]), torch.stack([v[1] for v in w])
    ids = torch.zeros(M, 1, dtype=torch.int32, device="cuda")
    plan = fq.fp8q_moe_plan(ids, E)
    q, sf = fq.fp8q_moe_fp4_quant(rnd(M, K, seed=80), plan, fmt)
    y = torch.full((2 * M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    wrong = plan._replace(offsets=torch.tensor([0, M + 40, 2 * M, -5, 1 << 30], dtype=torch.int32, device="cuda"),
                          sf_offsets=torch.tensor([0, 99, -3, 1 << 29, 7], dtype=torch.int32, device="cuda"))
    fq.fp8q_grouped_mm_fp4(q, b, sf, bsf, fmt, wrong, y=y[:M])
    assert fq.fp8q_last_device_status() == fq.OK and bool((y[M:] == 3).all())


def test_plans_and_rows_that_do_not_match_are_refused():
    E, K, fmt = 4, 128, "nvfp4"
    ids = torch.zeros(10, 2, dtype=torch.int32, device="cuda")
    plan = fq.fp8q_moe_plan(ids, E)
    x = rnd(10, K)
    q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
    w, wsf = torch.zeros(E, 64, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(
        E, *fq.fp4_sf_shape(64, K, fmt), dtype=torch.uint8, device="cuda")
    for bad in (lambda: fq.fp8q_moe_fp4_quant(x[:9], plan, fmt),
                lambda: fq.fp8q_grouped_mm_fp4(q[:19], w, sf, wsf, fmt, plan),
                lambda: fq.fp8q_grouped_mm_fp4(q, w[:3], sf, wsf[:3], fmt, plan),
                lambda: fq.fp8q_grouped_mm_fp4(q, w, sf[:1], wsf, fmt, plan),
                lambda: fq.fp8q_moe_combine(torch.zeros(19, 64, dtype=torch.bfloat16, device="cuda"), plan,
                                            torch.ones(10, 2, device="cuda")),
                lambda: fq.fp8q_moe_combine(torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda"), plan,
                                            torch.ones(10, 3, device="cuda")),
                lambda: fq.fp8q_moe_plan(ids, 0)):
        with pytest.raises((ValueError, fq.Fp8qError)):
            bad()


def test_arguments_that_are_refused_by_their_kind():
    l = torch.zeros(3, 8, device="cuda")
    for k in (0, -1):
        with pytest.raises(ValueError):
            fq.fp8q_moe_route(l, k)
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_route(torch.zeros(3, 64, device="cuda"), 33)
    with pytest.raises(ValueError):
        fq.fp8q_moe_plan(torch.zeros(3, 2, dtype=torch.int32, device="cuda"), -4)
    with pytest.raises(TypeError):
        fq.fp8q_moe_plan(torch.zeros(3, 2, dtype=torch.int64, device="cuda"), 4)
    w13, s13, w2, s2 = experts_weights(2, 64, 128, "nvfp4", 90)
    x, ids, w = rnd(3, 64), torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, 1, device="cuda")
    good = [x, ids, w, w13, s13, w2, s2, "nvfp4"]
    assert fq.fp8q_moe_experts_fp4(*good).shape == (3, 64)
    for at, bad in ((0, x.float()), (0, x.cpu()), (1, ids.long()), (1, ids.tolist()), (1, ids[0]), (2, w.half()), (2, w[:2]),
                    (3, w13[0]), (3, w13.float()), (4, s13[:1]), (5, w2.transpose(1, 2)), (6, s2.int()), (7, "fp4")):
        with pytest.raises((TypeError, ValueError)):
            fq.fp8q_moe_experts_fp4(*good[:at], bad, *good[at + 1:])


@pytest.mark.parametrize("fmt", FMTS)
def test_replayed_pairs_and_remainders_follow_their_inputs(fmt):
    """Experts of many rows (whole tiles and remainders in two launches), captured once: every replay
    on other ids, tokens and expert scales gives what a call gives."""
    T, E, N, K = 4000, 4, 1024, 256
    w = [fq.fp8q_fp4_quant(rnd(N, K, seed=300 + e), fmt) for e in range(E)]
    b, bsf = torch.stack([v[0] for v in w]), torch.stack([v[1] for v in w])
    x, ids = rnd(T, K, seed=310), torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    gb = torch.ones(E, device="cuda") if fmt == "nvfp4" else None

    def run():
        plan = fq.fp8q_moe_plan(ids, E)
        q, sf = fq.fp8q_moe_fp4_quant(x, plan, fmt)
        o = fq.fp8q_grouped_mm_fp4(q, b, sf, bsf, fmt, plan, b_gscale=gb)
        return fq.fp8q_moe_combine(o, plan, torch.ones(T, 1, device="cuda"))

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i in range(12):
        x.copy_(rnd(T, K, seed=320 + i))
        share = torch.rand(E, device="cuda", generator=gen) + 0.01
        ids.copy_(torch.multinomial(share, T, replacement=True, generator=gen).int().view(T, 1))
        if gb is not None:
            gb.copy_(torch.rand(E, device="cuda", generator=gen) + 0.5)
        for _ in range(2):
            graph.replay()
        got = y.clone()
        assert torch.equal(got, run())
        # row by row: a token's row depends on its expert alone
        for e in range(E):
            rows = torch.nonzero(ids[:, 0] == e)[:100, 0]
            if len(rows):
                q, sf = fq.fp8q_fp4_quant(x[rows], fmt)
                d = fq.fp8q_scaled_mm_fp4(q, b[e], sf, bsf[e], fmt, b_gscale=None if gb is None else gb[e:e + 1]).double()
                # the same products in another order: fp32 accumulation, then a rounding to bf16
                assert bool(((got[rows].double() - d).abs() <= 2.0 ** -6 * d.abs() + 2.0 ** -12 * d.abs().mean()).all())
    assert fq.fp8q_last_device_status() == fq.OK


@pytest.mark.parametrize("n,E", [(8192, 512), (28673, 3), (32768, 500), (32769, 64), (45000, 512), (300000, 128)])
def test_plan_of_many_entries(n, E):
    """Both sides of a plan whose blocks are one cluster, back to back on other ids."""
    rng = np.random.default_rng(n)
    for _ in range(3):
        ids = rng.integers(-1, E + 1, (n, 1)).astype(np.int32)
        p = fq.fp8q_moe_plan(torch.from_numpy(ids).cuda(), E)
        for got, want, name in zip(p, fp4.plan(ids, E), p._fields):
            np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
