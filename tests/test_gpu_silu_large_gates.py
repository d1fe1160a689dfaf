"""SiLU*mul quantization of gates so large that gate * log2(e) leaves fp32:
silu(g) = g there, and the value may be ordinary (a tiny up), large or infinite."""
import numpy as np
import pytest
import torch

import fp8q_inputs as inp
import oracle
from helpers import assert_fused_quant_close, codes_np, to_dev_bf16
from oracle import fp4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq

# either side of 85, of 2^127 and of fl32's largest / log2 e (2.3587e38, between two bf16 values)
GATES = np.array([84.5, 85.5, 88, 100, 1e4, 1e30, 1.6e38, 1.7014118e38, 1.8e38, 2.35e38, 2.36e38, 2.38e38, 3e38,
                  3.3895e38], np.float32)


def gates_and_ups(M, I, infinite):
    """Ordinary rows with large gates here and there, rows of them alone, and (if `infinite`) gates of
    +inf and products that overflow; ups of both signs that bring the values back to ordinary ones."""
    rng = np.random.default_rng(71)
    gate, up = rng.standard_normal((2, M, I)).astype(np.float32)
    at = rng.random((M, I)) < 0.04
    at[M // 2:] |= rng.random((M - M // 2, I)) < 0.9
    gate[at] = rng.choice(GATES, int(at.sum()))
    up[at] /= gate[at]                                                # values of about 1, some of subnormal ups
    if infinite:
        gate[1, 5] = gate[M - 1, 9] = gate[M // 2, ::16] = np.inf      # groups with one infinity, of either sign
        up[1, 5], up[M - 1, 9], up[M // 2, ::32], up[M // 2, 16::32] = 1e-38, -2.0, -3.0, 1.5
        gate[2, 8], up[2, 8] = 3e38, 7.0                               # overflows
        gate[3, 40:48], up[3, 40:48] = 2.4e38, -1e20
    return inp.to_bf16_bits(np.concatenate([gate, up], 1))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_fp4(fmt):
    M, I = 64, 288
    x = gates_and_ups(M, I, True)
    v = inp.bf16_bits_to_f32(x).astype(np.float64)
    y = fp4.bf16(fp4.silu_mul(v[:, :I], v[:, I:]))
    assert not np.isnan(y).any()
    for g in (None, 0.0371, 2.0 ** 40) if fmt == "nvfp4" else (None,):
        gs = None if g is None else torch.tensor([g], device="cuda")
        q, sf = fq.fp8q_silu_mul_fp4_quant(to_dev_bf16(x), fmt, gscale=gs)
        codes, b = fp4.quantize(y, fmt, 1.0 if g is None else float(np.float32(g)))
        np.testing.assert_array_equal(fp4.load_scales(sf.cpu().numpy(), M, b.shape[1]), b)
        np.testing.assert_array_equal(fp4.unpack(q.cpu().numpy()), codes)


@pytest.mark.parametrize("exact", [0, 1])
@pytest.mark.parametrize("per_token", [False, True])
def test_fp8(per_token, exact):
    M, I = 64, 256
    x = gates_and_ups(M, I, False)
    g = I if per_token else 128
    q_ref, s_ref = oracle.silu_mul_quant(x, g)
    before = fq.fp8q_get_fused_quant_exact()
    fq.fp8q_set_fused_quant_exact(exact)
    try:
        q, s = fq.fp8q_silu_mul_quant(to_dev_bf16(x), g)
        torch.cuda.synchronize()
    finally:
        fq.fp8q_set_fused_quant_exact(before)
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    if exact or not per_token:
        np.testing.assert_array_equal(codes_np(q), q_ref)
    else:
        assert_fused_quant_close(codes_np(q), s.cpu().numpy(), q_ref, s_ref, "large gates")


def test_i8():
    M, I = 64, 256
    x = gates_and_ups(M, I, False)
    q_ref, s_ref = oracle.silu_mul_quant_i8(x, I)
    before = fq.fp8q_get_fused_quant_exact()
    fq.fp8q_set_fused_quant_exact(1)
    try:
        q, s = fq.fp8q_silu_mul_quant_i8(to_dev_bf16(x), I)
        torch.cuda.synchronize()
    finally:
        fq.fp8q_set_fused_quant_exact(before)
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref)
