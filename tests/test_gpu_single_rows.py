"""A single row's stride means nothing: the 4-bit operators and the experts take
it from any view, as decode steps cut it out of a batch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq


def odd(t, stride):
    """The same single row with another row stride."""
    assert t.shape[0] == 1
    return torch.as_strided(t, t.shape, (stride, 1))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("stride", [0, 1, 7, 1001])
def test_single_rows(fmt, stride):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    H, I, E, k = 256, 128, 4, 2
    x, w = rnd(1, H), rnd(H)
    xs = odd(x, stride)
    for got, want in zip(fq.fp8q_fp4_quant(xs, fmt), fq.fp8q_fp4_quant(x, fmt)):
        assert torch.equal(got[..., :4], want[..., :4])
    q, sf = fq.fp8q_rmsnorm_fp4_quant(x, w, 1e-6, fmt)
    assert torch.equal(fq.fp8q_rmsnorm_fp4_quant(xs, w, 1e-6, fmt)[0], q)
    assert torch.equal(fq.fp8q_silu_mul_fp4_quant(xs, fmt)[0], fq.fp8q_silu_mul_fp4_quant(x, fmt)[0])
    out = odd(torch.zeros_like(q), stride)
    fq.fp8q_rmsnorm_fp4_quant(x, w, 1e-6, fmt, q=out)
    assert torch.equal(out, q)
    v = fq.fp8q_fp4_dequant(q, sf, fmt)
    y = odd(torch.zeros_like(v), stride)
    assert torch.equal(fq.fp8q_fp4_dequant(odd(q, stride), sf, fmt, y=y), v)
    b, bsf = fq.fp8q_fp4_quant(rnd(H, H), fmt)
    y.zero_()
    assert torch.equal(fq.fp8q_scaled_mm_fp4(q, b, sf, bsf, fmt, y=y), fq.fp8q_scaled_mm_fp4(q, b, sf, bsf, fmt))
    w13, s13, w2, s2 = (torch.stack(t) for shape in ((2 * I, H), (H, I))
                        for t in zip(*(fq.fp8q_fp4_quant(rnd(*shape), fmt) for _ in range(E))))
    wt, ids = fq.fp8q_moe_route(odd(torch.randn(1, E, device="cuda", generator=g), stride), k)
    want = fq.fp8q_moe_experts_fp4(x, ids, wt, w13, s13, w2, s2, fmt)
    y.zero_()
    assert torch.equal(fq.fp8q_moe_experts_fp4(xs, ids, wt, w13, s13, w2, s2, fmt, y=y), want)
    plan = fq.fp8q_moe_plan(ids[:, :1].contiguous(), E)
    for got, like in zip(fq.fp8q_moe_fp4_quant(xs, plan, fmt), fq.fp8q_moe_fp4_quant(x, plan, fmt)):
        assert torch.equal(got.view(-1)[:4], like.view(-1)[:4])
    one = wt[:, :1].contiguous()
    assert torch.equal(fq.fp8q_moe_combine(xs, plan, one, y=y), fq.fp8q_moe_combine(x, plan, one))
    assert fq.fp8q_last_device_status() == fq.OK
    # several rows keep their rule
    for bad in (0, 7, H - 8):
        with pytest.raises(fq.Fp8qError):
            fq.fp8q_fp4_quant(torch.as_strided(rnd(8, H), (3, H), (bad, 1)), fmt)
