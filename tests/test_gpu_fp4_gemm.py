"""The 4-bit block-scaled GEMM against an fp64 product of the same codes.

Tolerance, from the arithmetic: one rounding to bf16 (half a step, 2^-8
relative at most), and the fp32 accumulation -- every 64-deep step adds its 64
exact products with at least 24 bits below the largest term, then the running
sum: at most (K / 64) 2^-23 + 64 2^-24 of the sum of absolute products.  The
tensor scales add two fp32 roundings (2^-23)."""
import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq

FMTS = ["nvfp4", "mxfp4"]


def operand(seed, rows, K, fmt, pad=0):
    """Random codes and scales: (packed codes, scale blocks, fp64 values); `pad` fills the scale
    bytes of rows that only complete the last block."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, K), dtype=np.uint8)
    lo, hi = (0, 127) if fmt == "nvfp4" else (120, 134)
    b = rng.integers(lo, hi, (rows, K // fp4.GROUP[fmt]), dtype=np.uint8)
    return (torch.from_numpy(fp4.pack(codes)).cuda(), torch.from_numpy(fp4.store_scales(b, pad)).cuda(),
            torch.from_numpy(fp4.values(codes, b, fmt)).cuda())


def check(y, a, b, K, alpha=1.0):
    ref = a @ b.t() * alpha
    absdot = a.abs() @ b.abs().t() * alpha
    tol = (2.0 ** -8 + 2.0 ** -22) * ref.abs() + ((K / 64) * 2.0 ** -23 + 2.0 ** -18) * absdot
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max())} x tolerance"


SHAPES = [(1, 16, 32), (1, 128, 256), (2, 272, 96), (16, 64, 544), (17, 512, 1024), (32, 80, 64), (33, 336, 288),
          (64, 4096, 512), (65, 400, 1056), (127, 144, 160), (128, 256, 2048), (129, 1040, 320), (200, 9600, 256),
          (300, 2576, 4096), (1000, 10256, 128), (4100, 5136, 224), (1, 5120, 25600), (8, 10240, 5120)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(fmt, M, N, K):
    # the bytes of absent rows hold NaN scales: they must not reach a result
    a, asf, av = operand(M + 7 * K, M, K, fmt, 0xFF)
    b, bsf, bv = operand(N + 5 * K, N, K, fmt, 0xFF)
    y = torch.full((M + 1, N + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, fmt, y=y[:M, :N])
    assert fq.fp8q_last_device_status() == fq.OK
    check(y[:M, :N], av, bv, K)
    assert bool((y[M] == 3).all()) and bool((y[:, N:] == 3).all())     # nothing written beside the result


@pytest.mark.parametrize("M", [1, 40, 300])
def test_tensor_scales(M):
    a, asf, av = operand(1, M, 512, "nvfp4")
    b, bsf, bv = operand(2, 528, 512, "nvfp4")
    g = [torch.tensor([v], device="cuda") for v in (0.0371, 0.00113)]
    check(fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, "nvfp4", a_gscale=g[0], b_gscale=g[1]), av, bv, 512,
          float(g[0].double() * g[1].double()))
    check(fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, "nvfp4", b_gscale=g[1]), av, bv, 512, float(g[1].double()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 100, 513])
def test_identity_weight_finds_every_column(fmt, M):
    """One-hot weights: each output is one code of the input times its scale, exactly (bf16 holds
    it), so that a swapped column, group or scale cannot hide."""
    K = N = 512
    a, asf, av = operand(3, M, K, fmt)
    codes = np.zeros((N, K), np.uint8)
    codes[np.arange(N), (np.arange(N) * 37) % K] = 2                   # 1.0
    b = np.full((N, K // fp4.GROUP[fmt]), 0x38 if fmt == "nvfp4" else 127, np.uint8)
    y = fq.fp8q_scaled_mm_fp4(a, torch.from_numpy(fp4.pack(codes)).cuda(), asf, torch.from_numpy(fp4.store_scales(b)).cuda(), fmt)
    assert torch.equal(y.double(), av[:, (torch.arange(N, device="cuda") * 37) % K])


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_do_not_depend_on_each_other(fmt):
    """A token's result is the same bits alone and in any batch of the same tile width, and on
    every run."""
    b, bsf, _ = operand(4, 4096, 1024, fmt)
    a, asf, _ = operand(5, 16, 1024, fmt)
    y = fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, fmt)
    for _ in range(3):
        assert torch.equal(fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, fmt), y)
    assert torch.equal(fq.fp8q_scaled_mm_fp4(a[:1], b, asf, bsf, fmt), y[:1])


@pytest.mark.parametrize("fmt", FMTS)
def test_e8m0_nan_stays_in_its_row(fmt):
    a, asf, _ = operand(6, 40, 256, fmt)
    b, bsf, _ = operand(7, 64, 256, fmt)
    asf[0, 0, 3 * 16] = 0xFF if fmt == "mxfp4" else 0x7F               # row 3, group 0
    y = fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, fmt)
    nan = y.isnan().any(dim=1).cpu().numpy()
    assert nan[3] and nan.sum() == 1


def test_linear_chain_and_graph():
    """RMSNorm quant -> gate_up -> SiLU*mul quant -> down, as a layer runs it, eager and from a
    graph replayed on new inputs; two graphs may be replayed in turn."""
    H, I, M = 512, 640, 48
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    w = rnd(H)
    for fmt in FMTS:
        w13, w2 = fq.fp8q_fp4_quant(rnd(2 * I, H), fmt), fq.fp8q_fp4_quant(rnd(H, I), fmt)

        def layer(x):
            q, sf = fq.fp8q_rmsnorm_fp4_quant(x, w, 1e-6, fmt)
            h = fq.fp8q_scaled_mm_fp4(q, w13[0], sf, w13[1], fmt)
            q, sf = fq.fp8q_silu_mul_fp4_quant(h, fmt)
            return fq.fp8q_scaled_mm_fp4(q, w2[0], sf, w2[1], fmt)

        x = rnd(M, H)
        layer(x)
        graphs = []
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                y = layer(x)
            graphs.append((gr, y))
        for _ in range(3):
            x.copy_(rnd(M, H))
            want = layer(x)
            for gr, y in graphs:
                y.zero_()
                gr.replay()
                assert torch.equal(y, want)
        # the layer against its parts dequantized in fp64
        q, sf = fq.fp8q_rmsnorm_fp4_quant(x, w, 1e-6, fmt)
        h = fq.fp8q_scaled_mm_fp4(q, w13[0], sf, w13[1], fmt)
        check(h, fq.fp8q_fp4_dequant(q, sf, fmt).double(), fq.fp8q_fp4_dequant(*w13, fmt).double(), H)


def test_refusals():
    a, asf, _ = operand(8, 16, 128, "nvfp4")
    b, bsf, _ = operand(9, 64, 128, "nvfp4")
    with pytest.raises(ValueError):
        fq.fp8q_scaled_mm_fp4(a, b[:, :32], asf, bsf, "nvfp4")
    with pytest.raises(ValueError):
        fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, "mxfp4")                 # blocks of the other format
    with pytest.raises(ValueError):
        fq.fp8q_scaled_mm_fp4(a, b, asf, bsf, "nvfp4", y=torch.empty(16, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        fq.fp8q_scaled_mm_fp4(a, b, asf.view(torch.int8), bsf, "nvfp4")
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_scaled_mm_fp4(a, b[:40].contiguous(), asf, bsf, "nvfp4")   # N not a multiple of 16
    assert fq.fp8q_scaled_mm_fp4(a[:0], b, asf[:0], bsf, "nvfp4").shape == (0, 64)
