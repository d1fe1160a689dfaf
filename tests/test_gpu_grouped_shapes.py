"""Shapes that the grouped products refuse."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N", [255, 257, 511])
def test_gate_up_rows_must_pair(fmt, N):
    """An odd number of weight rows has no halves: taken as one less, every expert after the first
    would begin a row too early."""
    E, K = 2, 128
    ids = torch.arange(6, dtype=torch.int32, device="cuda").view(6, 1) % E
    plan = fq.fp8q_moe_plan(ids, E)
    q, sf = fq.fp8q_moe_fp4_quant(torch.ones(6, K, dtype=torch.bfloat16, device="cuda"), plan, fmt)
    b = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    bsf = torch.zeros(E, *fq.fp4_sf_shape(N, K, fmt), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        fq.fp8q_grouped_mm_fp4_silu_quant(q, b, sf, bsf, fmt, plan)
    b = torch.zeros(E, 256, K // 2, dtype=torch.uint8, device="cuda")
    bsf = torch.zeros(E, *fq.fp4_sf_shape(256, K, fmt), dtype=torch.uint8, device="cuda")
    h, _ = fq.fp8q_grouped_mm_fp4_silu_quant(q, b, sf, bsf, fmt, plan)
    assert h.shape == (6, 64) and not bool((h & 0x77).any())           # zero weights: codes of zero
