"""4-bit quantization and dequantization against the fp64 oracle: codes and
scale bytes equal bit for bit (every rounding is part of the definition)."""
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


def gpu_g(g):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")


def f32_of(g):
    return 1.0 if g is None else float(np.float32(g))


def check(q, sf, y, fmt, g):
    """Codes and the scale bytes of the rows that exist (and the zeroed group padding)."""
    M, K = y.shape
    codes, b = fp4.quantize(y, fmt, f32_of(g))
    got = sf.cpu().numpy()
    np.testing.assert_array_equal(fp4.load_scales(got, M, b.shape[1]), b)
    np.testing.assert_array_equal(fp4.unpack(q.cpu().numpy()), codes)
    kb = -(-b.shape[1] // 4)
    pad = fp4.load_scales(got.reshape(-1), M, 4 * kb)[:, b.shape[1]:]
    assert not pad.any()


def values(bits):
    return inp.bf16_bits_to_f32(bits).astype(np.float64)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,ld", [(1, 32, 32), (1, 4096, 4096), (3, 96, 104), (129, 544, 552), (300, 5120, 6144),
                                    (64, 160, 176), (257, 32, 48)])
def test_plain(fmt, M, K, ld):
    x = inp.heavy_tailed_bf16(11 + K, M, K)
    for g in (None, 0.0371, 2.0 ** -7) if fmt == "nvfp4" else (None,):
        sf = torch.full(fq.fp4_sf_shape(M, K, fmt), 0xA5, dtype=torch.uint8, device="cuda")
        q = torch.full((M, K // 2 + 8), 0x5A, dtype=torch.uint8, device="cuda")[:, :K // 2]
        fq.fp8q_fp4_quant(to_dev_bf16(x, ld=ld), fmt, gscale=gpu_g(g), q=q, sf=sf)
        check(q, sf, values(x), fmt, g)
        # rows behind the last one stay as they were
        rows = fp4.load_scales(sf.cpu().numpy(), sf.shape[0] * 128, sf.shape[1] * 4)[M:]
        assert (rows == 0xA5).all() and (q.untyped_storage().nbytes() == M * (K // 2 + 8))
        assert bool((torch.as_strided(q, (M, 8), (K // 2 + 8, 1), K // 2) == 0x5A).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_special_values(fmt):
    """Zeros of both signs, groups of zeros, subnormals, the largest values, infinities, and
    quotients that lie exactly on a rounding border."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 256)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, ::2] = -0.0
    x[3] = 1e-40
    x[4] *= np.float32(1e-38)
    x[5] *= np.float32(3e37)
    x[6, 7] = np.inf
    x[7, 200] = -np.inf
    x[8, :32], x[8, 32:64] = 3.3895e38, 1e-10
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    for r in range(9, 40):                      # scales 2^k: values on the borders and a step beside them
        x[r] = np.tile(grid, 32) * np.float32(2.0 ** (r - 20)) * np.where(np.arange(256) % 3, 1, -1)
    x[25:40:2] *= np.float32(1 + 2.0 ** -7)
    bits = inp.to_bf16_bits(x)
    for g in (None, 0.125, 0.3) if fmt == "nvfp4" else (None,):
        q, sf = fq.fp8q_fp4_quant(to_dev_bf16(bits), fmt, gscale=gpu_g(g))
        check(q, sf, values(bits), fmt, g)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,H", [(1, 32), (1, 4096), (7, 5120), (130, 96), (33, 12288), (3, 25600), (2, 32768 + 96),
                                 (65, 608)])
def test_rmsnorm(fmt, M, H):
    x, w = inp.heavy_tailed_bf16(21 + H, M, H), inp.rms_weight_bf16(22, H)
    y = fp4.rmsnorm(values(x), values(w), 1e-6)
    for g in (None, 0.0071) if fmt == "nvfp4" else (None,):
        q, sf = fq.fp8q_rmsnorm_fp4_quant(to_dev_bf16(x, ld=H + 8), to_dev_bf16(w[None])[0], 1e-6, fmt, gscale=gpu_g(g))
        check(q, sf, y, fmt, g)


def test_rmsnorm_zero_rows_and_eps():
    x = np.zeros((3, 64), np.uint16)
    w = inp.rms_weight_bf16(23, 64)
    for eps in (0.0, 1e-6):
        q, sf = fq.fp8q_rmsnorm_fp4_quant(to_dev_bf16(x), to_dev_bf16(w[None])[0], eps, "nvfp4")
        if eps:
            check(q, sf, np.zeros((3, 64)), "nvfp4", None)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,I,ld", [(1, 32, 64), (5, 12288, 24576), (131, 416, 840), (64, 1024, 2064)])
def test_silu_mul(fmt, M, I, ld):
    x = inp.heavy_tailed_bf16(31 + I, M, 2 * I)
    v = values(x)
    y = fp4.bf16(fp4.silu_mul(v[:, :I], v[:, I:]))
    for g in (None, 0.0371) if fmt == "nvfp4" else (None,):
        q, sf = fq.fp8q_silu_mul_fp4_quant(to_dev_bf16(x, ld=ld), fmt, gscale=gpu_g(g))
        check(q, sf, y, fmt, g)


@pytest.mark.parametrize("fmt", FMTS)
def test_silu_mul_of_very_negative_gates(fmt):
    """Gates at both sides of -60 and -85 and far below, beside ordinary ones and filling whole
    groups (whose scale, with a small tensor scale, they then decide), with ups of every size."""
    rng = np.random.default_rng(17)
    M, I = 96, 256
    gate = rng.standard_normal((M, I)).astype(np.float32)
    up = rng.standard_normal((M, I)).astype(np.float32)
    odd = np.array([-59.75, -60, -60.25, -61, -84.5, -85, -85.5, -88, -89, -100, -1e4, -3e38], np.float32)
    at = rng.random((M, I)) < 0.05
    gate[at] = rng.choice(odd, at.sum())
    gate[32:64] = rng.uniform(-75, -45, (32, I))                       # small groups
    gate[64:80] = rng.choice(odd, (16, I))
    up[40:72] *= np.float32(2.0) ** rng.integers(-60, 90, (32, I))
    up[80:] *= np.float32(1e30)
    up[3, ::7], up[4, ::7], up[5, ::5] = 0.0, -0.0, 1e-30
    up[6, 3], up[7, 3], up[66, 9] = np.inf, -np.inf, np.inf
    gate[6, 3] = gate[7, 3] = gate[66, 9] = -70
    x = inp.to_bf16_bits(np.concatenate([gate, up], 1))
    v = values(x)
    y = fp4.bf16(fp4.silu_mul(v[:, :I], v[:, I:]))
    for g in (None, 2.0 ** -60, 2.0 ** 40) if fmt == "nvfp4" else (None,):
        q, sf = fq.fp8q_silu_mul_fp4_quant(to_dev_bf16(x), fmt, gscale=gpu_g(g))
        check(q, sf, y, fmt, g)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 32), (130, 608), (1000, 4096)])
def test_dequant(fmt, M, K):
    rng = np.random.default_rng(41)
    codes = rng.integers(0, 16, (M, K), dtype=np.uint8)
    b = rng.integers(0, 127 if fmt == "nvfp4" else 255, (M, K // fp4.GROUP[fmt]), dtype=np.uint8)
    if fmt == "mxfp4":
        b = np.clip(b, 8, 250)                 # bf16 holds these exactly
    for g in (None, 0.0371) if fmt == "nvfp4" else (None,):
        y = torch.full((M, K + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        fq.fp8q_fp4_dequant(torch.from_numpy(fp4.pack(codes)).cuda(), torch.from_numpy(fp4.store_scales(b, 0xFF)).cuda(),
                            fmt, gscale=gpu_g(g), y=y[:, :K])
        np.testing.assert_array_equal(y[:, :K].double().cpu().numpy(), fp4.dequant_bf16(codes, b, fmt, f32_of(g)))
        assert bool((y[:, K:] == 7).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_round_trip_of_values(fmt):
    """Quantizing what codes stand for gives them back."""
    x = to_dev_bf16(inp.normal_bf16(51, (257, 1056)))
    y = fq.fp8q_fp4_dequant(*fq.fp8q_fp4_quant(x, fmt), fmt)
    assert torch.equal(fq.fp8q_fp4_dequant(*fq.fp8q_fp4_quant(y, fmt), fmt), y) or fmt == "nvfp4"
    err = (y.double() - x.double()).norm() / x.double().norm()
    assert err < 0.25                          # at most half a step of e2m1 (2^-2) of each value, or of the least


def test_streams_and_zero_rows():
    x = to_dev_bf16(inp.normal_bf16(61, (64, 512)))
    want = fq.fp8q_fp4_quant(x, "nvfp4")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = fq.fp8q_fp4_quant(x, "nvfp4", stream=stream)
        s.synchronize()
        assert torch.equal(got[0], want[0])
    q, sf = fq.fp8q_fp4_quant(x[:0], "mxfp4")
    assert q.shape == (0, 256) and sf.shape == (0, 4, 512)
    with pytest.raises(ValueError):
        fq.fp8q_fp4_quant(x, "nvfp4", sf=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fq.fp8q_fp4_quant(x.t(), "nvfp4")
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_fp4_quant(x, "mxfp4", gscale=gpu_g(1.0))
