"""Ids of experts that are not here: whatever lies outside [0, num_experts) has
no row, the ids less a first expert (negative, any size) as well as -1 and E."""
import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_quantized_linear_rms_b200 as fq

LOWEST = -2 ** 31


def absent_ids(T, k, E, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "shifted":                      # 4 E experts over four GPUs, the third's here
        ids = rng.integers(0, 4 * E, (T, k)) - 2 * E
    elif kind == "wide":
        ids = rng.integers(-4 * E, 4 * E, (T, k))
    else:                                      # whatever shares an expert's low bits
        bits = max(1, int(E).bit_length())
        odd = [-E, -E - 1, -2 ** bits, -2 ** bits + E - 1, -200, LOWEST, LOWEST + E // 2, -1, E, 2 ** 31 - 1]
        ids = np.where(rng.random((T, k)) < 0.5, rng.integers(0, E, (T, k)), rng.choice(odd, (T, k)))
    return ids.astype(np.int32)


@pytest.mark.parametrize("kind", ["shifted", "wide", "odd"])
@pytest.mark.parametrize("T,k,E", [(3, 4, 16), (40, 3, 16), (300, 4, 16), (150, 8, 128), (1000, 1, 1), (2000, 2, 512),
                                   (4000, 8, 64), (9000, 4, 33)])      # one block, one cluster, more blocks
def test_plan_of_absent_ids(T, k, E, kind):
    ids = absent_ids(T, k, E, kind, T + E)
    p = fq.fp8q_moe_plan(torch.from_numpy(ids).cuda(), E)
    for got, want, name in zip(p, fp4.plan(ids, E), p._fields):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)


@pytest.mark.parametrize("kind", ["shifted", "wide", "odd"])
@pytest.mark.parametrize("T,k", [(3, 4), (32, 4), (33, 4), (500, 3)])  # both sides of 128 entries
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_experts_of_absent_ids(fmt, T, k, kind):
    """Absent ids by other names give the bits that -1 gives."""
    E, H, I = 16, 256, 128
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    w13, s13, w2, s2 = (torch.stack(t) for shape in ((2 * I, H), (H, I))
                        for t in zip(*(fq.fp8q_fp4_quant(rnd(*shape), fmt) for _ in range(E))))
    ids = absent_ids(T, k, E, kind, T)
    plain = np.where((ids >= 0) & (ids < E), ids, -1).astype(np.int32)
    x, w = rnd(T, H), torch.rand(T, k, device="cuda", generator=g)
    y, want = (fq.fp8q_moe_experts_fp4(x, torch.from_numpy(i).cuda(), w, w13, s13, w2, s2, fmt) for i in (ids, plain))
    assert fq.fp8q_last_device_status() == fq.OK
    assert torch.equal(y, want) and bool(want.any())
    none = torch.from_numpy((plain >= 0).any(1)).cuda().logical_not()
    assert not bool(y[none].any())                                     # a token without an expert here
