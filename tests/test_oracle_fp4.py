"""Pins of the 4-bit oracle (oracle/fp4.py): formats against ml_dtypes, the
quantizer's invariants, the scale layout, routing by hand, and the plan."""
import ml_dtypes
import numpy as np
import pytest

from oracle import fp4


def test_e2m1_codes():
    fmt = ml_dtypes.float4_e2m1fn
    assert np.array_equal(fp4.e2m1_decode(np.arange(16)), np.arange(16, dtype=np.uint8).view(fmt).astype(np.float64))
    v = np.concatenate([np.linspace(-7, 7, 5601), np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])])
    assert np.array_equal(fp4.e2m1_encode(v), v.astype(np.float32).astype(fmt).view(np.uint8) & 15)
    # ties to the even code, saturation, signed zeros
    assert fp4.e2m1_encode([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 9, np.inf]).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    assert fp4.e2m1_encode([-0.0, -0.2, -5.1]).tolist() == [8, 8, 15]


def test_e4m3_scales():
    b = np.arange(127, dtype=np.uint8)
    assert np.array_equal(fp4.e4m3_decode(b), b.view(ml_dtypes.float8_e4m3fn).astype(np.float64))
    assert np.array_equal(fp4.e4m3_encode(fp4.e4m3_decode(b)), b)
    v = np.exp(np.random.default_rng(1).uniform(np.log(2.0 ** -12), np.log(448), 20000)).astype(np.float32)
    assert np.array_equal(fp4.e4m3_encode(v), v.astype(ml_dtypes.float8_e4m3fn).view(np.uint8))
    assert fp4.e4m3_encode([1e9, np.inf, 2.0 ** -10, 0.0]).tolist() == [126, 126, 0, 0]


def test_bf16_rounding():
    v = np.random.default_rng(2).standard_normal(20000).astype(np.float32)
    assert np.array_equal(fp4.bf16(v), v.astype(ml_dtypes.bfloat16).astype(np.float64))
    assert fp4.bf16(1 + 2.0 ** -8 + 2.0 ** -30) == 1 + 2.0 ** -7     # one rounding only


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantizer_invariants(fmt):
    rng = np.random.default_rng(3)
    y = fp4.bf16(rng.standard_normal((64, 96)) * np.exp(rng.uniform(-3, 3, (64, 1))))
    y[5, :32] = 0
    codes, b = fp4.quantize(y, fmt)
    back = fp4.values(codes, b, fmt)
    s = np.repeat(fp4.scale_values(b, fmt), fp4.GROUP[fmt], axis=1)
    amax = np.repeat(np.abs(y).reshape(64, -1, fp4.GROUP[fmt]).max(2), fp4.GROUP[fmt], axis=1)
    # half of the widest step (2) times the scale, and what saturation cuts off: an e4m3 scale may lie
    # half a step (2^-4) below amax / 6
    assert np.all(np.abs(back - y) <= s * (1 + 6 * 2.0 ** -4) + 1e-30)
    assert np.all(back[5, :32] == 0)
    if fmt == "mxfp4":
        assert np.all(s >= np.maximum(amax, 1e-10) / 6 * (1 - 2.0 ** -23)) and np.all(s < np.maximum(amax, 1e-10) / 3)
        assert b[5, 0] == 127 - 35             # fl32(1e-10 / 6) lies in (2^-36, 2^-35)
    else:
        assert b[5, 0] == 0
    # a tensor scale that is a power of two moves into the group scales, where they stay normal
    if fmt == "nvfp4":
        c2, b2 = fp4.quantize(y, fmt, 0.25)
        same = np.repeat((b > 8) & (b2 < 126), 16, axis=1)   # 8 may be rounded up from a subnormal
        assert same.any() and np.array_equal(c2[same], codes[same])


def test_hand_cases():
    y = np.zeros((1, 32))
    y[0, :4] = [6.0, -3.0, 1.25, 0.5]
    c, b = fp4.quantize(y, "nvfp4")            # sf = 1
    assert b.tolist() == [[0x38, 0]] and c[0, :4].tolist() == [7, 13, 2, 1]
    c, b = fp4.quantize(y, "mxfp4")
    assert b.tolist() == [[127]] and c[0, :4].tolist() == [7, 13, 2, 1]
    y[0, 0] = 6.03125                          # just above: the power of two doubles
    assert fp4.quantize(y, "mxfp4")[1].tolist() == [[128]]


def test_scale_layout():
    b = np.random.default_rng(4).integers(0, 127, (300, 7), dtype=np.uint8)
    s = fp4.store_scales(b)
    assert s.shape == (3, 2, 512) and np.array_equal(fp4.load_scales(s, 300, 7), b)
    assert s[1, 1, 5 * 16 + 2 * 4 + 1] == b[128 + 64 + 5, 5]
    assert np.array_equal(fp4.unpack(fp4.pack((b & 15)[:, :6])), (b & 15)[:, :6])


def test_route_by_hand():
    l = np.array([[1.0, 3.0, 3.0, -np.inf, np.nan, 0.0]])
    w, i = fp4.route(l, 3, "softmax")
    assert i.tolist() == [[1, 2, 0]] and np.allclose(w.sum(), 1)       # equal logits: lowest index first
    w, i = fp4.route(l, 6, "softmax", renorm=False)
    assert i.tolist() == [[1, 2, 0, 5, 3, 4]] and w[0, 4] == w[0, 5] == 0
    w, i = fp4.route(np.full((1, 6), -np.inf), 2, "softmax")
    assert i.tolist() == [[0, 1]] and w.tolist() == [[0, 0]]
    # groups of two, one kept: with a bias by the sum of both, without by the larger
    l = np.array([[5.0, -5.0, 4.0, 3.9]])
    assert fp4.route(l, 1, "sigmoid", groups=2, topg=1)[1].tolist() == [[0]]
    assert fp4.route(l, 1, "sigmoid", bias=np.zeros(4), groups=2, topg=1)[1].tolist() == [[2]]


def test_plan_by_hand():
    ids = np.array([[2, 0], [2, 5], [-1, 0]], np.int32)
    off, sf, pos, row = fp4.plan(ids, 4)
    assert off.tolist() == [0, 2, 2, 4, 4] and sf.tolist() == [0, 1, 1, 2, 2]
    assert pos.tolist() == [[2, 0], [3, -1], [-1, 1]] and row.tolist() == [[128, 0], [129, -1], [-1, 1]]
