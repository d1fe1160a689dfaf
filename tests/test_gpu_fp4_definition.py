"""4-bit quantization against the fp64 oracle, bit for bit, over thousands of rows of heavy-tailed
values: enough of them next to a rounding border of y (one in some 40000 lies where rounding twice,
through fp32, would give another bf16 value) that a kernel which decides those another way is seen.
And what the smaller tests leave open: quantizing values that are quantized already, eps = 0."""
import numpy as np
import pytest
import torch

import fp8q_inputs as inp
from helpers import to_dev_bf16
from oracle import fp4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq

FMTS = ["nvfp4", "mxfp4"]


def values(bits):
    return inp.bf16_bits_to_f32(bits).astype(np.float64)


def check(q, sf, y, fmt, g=None):
    codes, b = fp4.quantize(y, fmt, 1.0 if g is None else float(np.float32(g)))
    np.testing.assert_array_equal(fp4.load_scales(sf.cpu().numpy(), *b.shape), b)
    np.testing.assert_array_equal(fp4.unpack(q.cpu().numpy()), codes)


def rounded_twice(v):
    """fp64 -> fp32 -> bf16."""
    return fp4.bf16(np.asarray(v).astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt", FMTS)
def test_silu_mul_of_many_rows(fmt):
    M, I = 4096, 2048
    x = inp.heavy_tailed_bf16(91, M, 2 * I)
    v = values(x)
    exact = fp4.silu_mul(v[:, :I], v[:, I:])
    y = fp4.bf16(exact)
    assert (y != rounded_twice(exact)).sum() > 20                      # the inputs hold such values
    q, sf = fq.fp8q_silu_mul_fp4_quant(to_dev_bf16(x), fmt)
    check(q, sf, y, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_of_many_rows(fmt):
    M, H = 4096, 2048
    x, w = inp.heavy_tailed_bf16(92, M, H), inp.rms_weight_bf16(93, H)
    q, sf = fq.fp8q_rmsnorm_fp4_quant(to_dev_bf16(x), to_dev_bf16(w[None])[0], 1e-6, fmt)
    check(q, sf, fp4.rmsnorm(values(x), values(w), 1e-6), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantizing_quantized_values(fmt):
    """The second pass is the oracle's quantization of the first one's values; with E8M0 scales it
    gives the values back (an e4m3 scale of 6 d / 6 may be rounded to another, and a value with it)."""
    x = to_dev_bf16(inp.normal_bf16(94, (257, 1056)))
    for g in (None, 0.0371) if fmt == "nvfp4" else (None,):
        gs = None if g is None else torch.tensor([g], device="cuda")
        y = fq.fp8q_fp4_dequant(*fq.fp8q_fp4_quant(x, fmt, gscale=gs), fmt, gscale=gs)
        q, sf = fq.fp8q_fp4_quant(y, fmt, gscale=gs)
        check(q, sf, y.double().cpu().numpy(), fmt, g)
        if fmt == "mxfp4":
            assert torch.equal(fq.fp8q_fp4_dequant(q, sf, fmt), y)


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_without_eps(fmt):
    """eps = 0: a row of zeros has no r (its codes are open), the rows beside it do; nothing is
    written beside the codes and scales of the rows."""
    M, H = 9, 96
    x, w = inp.heavy_tailed_bf16(95, M, H), inp.rms_weight_bf16(96, H)
    x[4] = 0
    rows = [r for r in range(M) if r != 4]
    q = torch.full((M + 1, H // 2 + 8), 0x5A, dtype=torch.uint8, device="cuda")
    sf = torch.full(fq.fp4_sf_shape(M, H, fmt), 0xA5, dtype=torch.uint8, device="cuda")
    fq.fp8q_rmsnorm_fp4_quant(to_dev_bf16(x), to_dev_bf16(w[None])[0], 0.0, fmt, q=q[:M, :H // 2], sf=sf)
    codes, b = fp4.quantize(fp4.rmsnorm(values(x)[rows], values(w), 0.0), fmt)
    np.testing.assert_array_equal(fp4.unpack(q[:M, :H // 2].cpu().numpy())[rows], codes)
    got = fp4.load_scales(sf.cpu().numpy(), 128, sf.shape[1] * 4)
    np.testing.assert_array_equal(got[rows, :b.shape[1]], b)
    assert bool((q[M] == 0x5A).all()) and bool((q[:, H // 2:] == 0x5A).all()) and (got[M:] == 0xA5).all()
