"""The experts' pass refuses sizes that one of its launches would refuse before
any of them (no kernel runs: the addresses are never dereferenced)."""
import pytest

import fp8_quantized_linear_rms_b200 as fq

P = 1 << 20


@pytest.mark.parametrize("T,k,E,H,I", [(1 << 20, 32, 1, 32, 1 << 24),       # tiles of the gate_up product past 32 bits
                                       (1 << 20, 32, 1, 1 << 24, 128),      # of the down product
                                       (1 << 14, 32, 60, 32, 1 << 24)])
def test_more_tiles_than_32_bits_count(T, k, E, H, I):
    n = fq.lib.fp8q_moe_experts_fp4_workspace_bytes(T, k, E, H, I, 0)
    assert n > 0
    st = fq.lib.fp8q_moe_experts_fp4(P, T, H, P, P, k, E, H, I, 0, P, P, P, P, None, None, None, None, P, H, P, n, None)
    assert st == fq.ERR_INVALID_ARG
