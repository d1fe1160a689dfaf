"""Python binding of libfp8q, the B200 (sm_100a) FP8 W8A8 linear-layer path.

Argument marshalling only: every entry point takes torch CUDA tensors, checks
dtypes and shapes enough to pass the right pointers, and calls the C ABI of
``include/fp8q.h`` and ``include/fp8q_fp4.h`` with the current CUDA stream.
All arithmetic runs in the library's kernels; there is no CPU or PyTorch
fallback, and importing this package fails loudly if ``libfp8q.so`` is missing (build it with
``python fp8_quantized_linear_rms_b200/build.py``).

The names match the C ABI:
  fp8q_group_quant, fp8q_rmsnorm_quant, fp8q_add_rmsnorm_quant, fp8q_silu_mul_quant
                                                                (activation quant)
  fp8q_scaled_mm, fp8q_scaled_mm_blockwise, fp8q_scaled_mm_blockwise_e8m0,
  fp8q_scaled_mm_blockwise_silu_quant                           (scaled FP8 GEMMs)
  fp8q_fp4_quant, fp8q_rmsnorm_fp4_quant, fp8q_silu_mul_fp4_quant, fp8q_fp4_dequant,
  fp8q_scaled_mm_fp4                                            (4-bit nvfp4 / mxfp4)
  fp8q_moe_route, fp8q_moe_plan, fp8q_moe_fp4_quant, fp8q_grouped_mm_fp4,
  fp8q_grouped_mm_fp4_silu_quant, fp8q_moe_combine, fp8q_moe_experts_fp4  (experts)
  fp8q_workspace_bytes, fp8q_select_gemm_variant, fp8q_force_gemm_variant,
  fp8q_last_device_status, fp8q_status_string, fp8q_version
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8q.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp8q.h")
FP4_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp8q_fp4.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libfp8q.so not found at {LIB_PATH}; build it with "
                      "`python fp8_quantized_linear_rms_b200/build.py`")

lib = ctypes.CDLL(LIB_PATH)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = range(5)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class GemmVariant(ctypes.Structure):
    """fp8q_gemm_variant: swap_ab, split_k, block_n, cta_pair."""
    _fields_ = [("swap_ab", ctypes.c_int), ("split_k", ctypes.c_int), ("block_n", ctypes.c_int),
                ("cta_pair", ctypes.c_int)]

    def as_dict(self):
        return {"swap_ab": self.swap_ab, "split_k": self.split_k, "block_n": self.block_n,
                "cta_pair": self.cta_pair}


_SIGS = {
    "fp8q_group_quant": (_INT, [_P, _I64, _I64, _I64, _INT, _INT, _P, _I64, _P, _I64, _I64, _P]),
    "fp8q_rmsnorm_quant": (_INT, [_P, _P, ctypes.c_float, _I64, _I64, _I64, _INT, _INT, _P, _I64,
                                  _P, _I64, _I64, _P]),
    "fp8q_silu_mul_quant": (_INT, [_P, _I64, _I64, _I64, _INT, _INT, _P, _I64, _P, _I64, _I64,
                                   _P]),
    "fp8q_add_rmsnorm_quant": (_INT, [_P, _P, _P, ctypes.c_float, _I64, _I64, _I64, _I64, _INT, _INT,
                                      _P, _I64, _P, _I64, _I64, _P]),
    "fp8q_set_fused_quant_exact": (_INT, [_INT]),
    "fp8q_get_fused_quant_exact": (_INT, []),
    "fp8q_scaled_mm": (_INT, [_P, _P, _P, _INT, _P, _INT, _I64, _I64, _I64, _P, _I64, _P,
                              ctypes.c_size_t, _P]),
    "fp8q_scaled_mm_blockwise": (_INT, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _P, _I64,
                                        _P, ctypes.c_size_t, _P]),
    "fp8q_scaled_mm_blockwise_silu_quant": (_INT, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _INT,
                                                   _P, _I64, _P, _I64, _I64, _P]),
    "fp8q_scaled_mm_blockwise_e8m0": (_INT, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _P,
                                             _I64, _P, ctypes.c_size_t, _P]),
    "fp8q_scaled_mm_blockwise_noalloc": (_INT, [_P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _P,
                                                _I64, _P]),
    "fp8q_qk_norm_rope": (_INT, [_P, _I64, _I64, _INT, _INT, _INT, _INT, ctypes.c_float, _P, _P, _P,
                                 _I64, _P, _INT, _P]),
    "fp8q_group_quant_i8": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _I64, _P]),
    "fp8q_rmsnorm_quant_i8": (_INT, [_P, _P, ctypes.c_float, _I64, _I64, _I64, _INT, _P, _I64, _P,
                                     _I64, _I64, _P]),
    "fp8q_silu_mul_quant_i8": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _I64, _P]),
    "fp8q_scaled_mm_i8": (_INT, [_P, _P, _P, _INT, _P, _INT, _I64, _I64, _I64, _P, _I64, _P,
                                 ctypes.c_size_t, _P]),
    "fp8q_fp4_sf_bytes": (ctypes.c_size_t, [_I64, _I64, _INT]),
    "fp8q_fp4_quant": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _P, _I64, _P, _P]),
    "fp8q_silu_mul_fp4_quant": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _P, _I64, _P, _P]),
    "fp8q_rmsnorm_fp4_quant": (_INT, [_P, _P, ctypes.c_float, _I64, _I64, _I64, _INT, _P, _P, _I64, _P, _P]),
    "fp8q_fp4_dequant": (_INT, [_P, _I64, _P, _INT, _P, _I64, _I64, _P, _I64, _P]),
    "fp8q_scaled_mm_fp4": (_INT, [_P, _P, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _I64, _P]),
    "fp8q_moe_route": (_INT, [_P, _INT, _I64, _I64, _I64, _INT, _INT, _P, _INT, _INT, _INT, ctypes.c_float,
                              _P, _P, _P]),
    "fp8q_moe_plan_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "fp8q_moe_plan": (_INT, [_P, _I64, _I64, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "fp8q_moe_fp4_quant": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _P, _INT, _P, _P, _I64, _P, _P]),
    "fp8q_grouped_mm_fp4": (_INT, [_P, _P, _P, _P, _INT, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64, _P]),
    "fp8q_grouped_mm_fp4_silu_quant": (_INT, [_P, _P, _P, _P, _INT, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P,
                                              _P, _P, _P]),
    "fp8q_moe_combine": (_INT, [_P, _I64, _P, _P, _I64, _INT, _I64, _P, _I64, _P]),
    "fp8q_moe_experts_fp4_workspace_bytes": (ctypes.c_size_t, [_I64, _INT, _I64, _I64, _I64, _INT]),
    "fp8q_moe_experts_fp4": (_INT, [_P, _I64, _I64, _P, _P, _INT, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _P, _I64, _P, ctypes.c_size_t, _P]),
    "fp8q_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _INT]),
    "fp8q_select_gemm_variant": (_INT, [_I64, _I64, _I64, _INT, ctypes.POINTER(GemmVariant)]),
    "fp8q_force_gemm_variant": (_INT, [ctypes.POINTER(GemmVariant)]),
    "fp8q_last_device_status": (_INT, [_P]),
    "fp8q_status_string": (ctypes.c_char_p, [_INT]),
    "fp8q_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class Fp8qError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {lib.fp8q_status_string(status).decode()} ({status})")


def header_functions(path: str = HEADER_PATH) -> list[str]:
    """Names of every function include/fp8q.h (or the header at `path`) declares."""
    with open(path) as f:
        text = f.read()
    return re.findall(r"^FP8Q_API\s+[\w\s\*]+?\b(fp8q_\w+)\s*\(", text, flags=re.M)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise Fp8qError(fn, status)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _rowmajor(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.stride(0)


def _ue8m0_mode(ue8m0) -> int:
    """False / True / "packed" -> the ABI's 0 (fp32) / 1 (power-of-two fp32) / 2 (E8M0 bytes)."""
    if ue8m0 == "packed":
        return 2
    if ue8m0 in (False, True, 0, 1):
        return int(ue8m0)
    raise ValueError(f"ue8m0 must be False, True or 'packed', got {ue8m0!r}")


def _scales_out(M, L, group, layout, device, scales, mode=0):
    G = L // group if group > 0 and L % group == 0 else 0
    dt = torch.uint8 if mode == 2 else torch.float32
    if scales is None:
        if layout == "group_major":
            scales = torch.empty((G, M), dtype=dt, device=device)
        else:
            scales = torch.empty((M, G), dtype=dt, device=device)
    elif scales.dtype != dt:
        raise TypeError(f"scales must be {dt} for ue8m0 mode {mode}")
    if layout == "group_major":
        return scales, 1, M
    return scales, G, 1


# --------------------------------------------------------------- activation quant
def fp8q_group_quant(x: torch.Tensor, group_size: int, ue8m0: bool = False, q=None, scales=None,
                     scale_layout: str = "row_major", stream=None):
    """per_token_group_fp8_quant (group_size=128) / per-token quant (group_size=K).

    x: bf16 [M, K].  Returns (q float8_e4m3fn [M, K], scales fp32 [M, K/g]
    (row_major) or [K/g, M] (group_major)).  ue8m0: False, True (power-of-two
    fp32 scales) or "packed" (the same scales as uint8 E8M0 bytes).
    """
    _need(x, torch.bfloat16, "x")
    ldx = _rowmajor(x, "x")
    M, K = x.shape
    mode = _ue8m0_mode(ue8m0)
    if q is None:
        q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    scales, ssm, ssg = _scales_out(M, K, group_size, scale_layout, x.device, scales, mode)
    st = lib.fp8q_group_quant(x.data_ptr(), M, K, ldx, group_size, mode, q.data_ptr(),
                              _rowmajor(q, "q"), scales.data_ptr(), ssm, ssg, _stream(stream))
    _check("fp8q_group_quant", st)
    return q, scales


def fp8q_rmsnorm_quant(x: torch.Tensor, w: torch.Tensor, eps: float, group_size: int,
                       ue8m0: bool = False, q=None, scales=None, scale_layout: str = "row_major",
                       stream=None):
    """rms_norm_dynamic_per_token_quant (group_size=H) / rms_norm_per_block_quant (128)."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    ldx = _rowmajor(x, "x")
    M, H = x.shape
    mode = _ue8m0_mode(ue8m0)
    if q is None:
        q = torch.empty((M, H), dtype=torch.float8_e4m3fn, device=x.device)
    scales, ssm, ssg = _scales_out(M, H, group_size, scale_layout, x.device, scales, mode)
    st = lib.fp8q_rmsnorm_quant(x.data_ptr(), w.data_ptr(), ctypes.c_float(eps), M, H, ldx,
                                group_size, mode, q.data_ptr(), _rowmajor(q, "q"),
                                scales.data_ptr(), ssm, ssg, _stream(stream))
    _check("fp8q_rmsnorm_quant", st)
    return q, scales


def fp8q_add_rmsnorm_quant(x: torch.Tensor, residual: torch.Tensor, w: torch.Tensor, eps: float,
                           group_size: int, ue8m0=False, q=None, scales=None,
                           scale_layout: str = "row_major", stream=None):
    """Residual add + RMSNorm quant: residual <- bf16(x + residual) in place, then
    rms_norm quant of the new residual.  Returns (q, scales)."""
    _need(x, torch.bfloat16, "x")
    _need(residual, torch.bfloat16, "residual")
    _need(w, torch.bfloat16, "w")
    ldx = _rowmajor(x, "x")
    ldr = _rowmajor(residual, "residual")
    M, H = x.shape
    if tuple(residual.shape) != (M, H):
        raise ValueError("residual must have x's shape")
    mode = _ue8m0_mode(ue8m0)
    if q is None:
        q = torch.empty((M, H), dtype=torch.float8_e4m3fn, device=x.device)
    scales, ssm, ssg = _scales_out(M, H, group_size, scale_layout, x.device, scales, mode)
    st = lib.fp8q_add_rmsnorm_quant(x.data_ptr(), residual.data_ptr(), w.data_ptr(), ctypes.c_float(eps),
                                    M, H, ldx, ldr, group_size, mode, q.data_ptr(), _rowmajor(q, "q"),
                                    scales.data_ptr(), ssm, ssg, _stream(stream))
    _check("fp8q_add_rmsnorm_quant", st)
    return q, scales


def fp8q_silu_mul_quant(x: torch.Tensor, group_size: int, ue8m0: bool = False, q=None,
                        scales=None, scale_layout: str = "row_major", stream=None):
    """silu_and_mul_dynamic_per_token_quant (group_size=I) / silu_and_mul_per_block_quant (128).

    x: bf16 [M, 2I] = [gate | up].
    """
    _need(x, torch.bfloat16, "x")
    ldx = _rowmajor(x, "x")
    M, I2 = x.shape
    I = I2 // 2
    mode = _ue8m0_mode(ue8m0)
    if q is None:
        q = torch.empty((M, I), dtype=torch.float8_e4m3fn, device=x.device)
    scales, ssm, ssg = _scales_out(M, I, group_size, scale_layout, x.device, scales, mode)
    st = lib.fp8q_silu_mul_quant(x.data_ptr(), M, I, ldx, group_size, mode, q.data_ptr(),
                                 _rowmajor(q, "q"), scales.data_ptr(), ssm, ssg, _stream(stream))
    _check("fp8q_silu_mul_quant", st)
    return q, scales


# --------------------------------------------------------------------- GEMMs
def fp8q_workspace_bytes(M: int, N: int, K: int, blockwise) -> int:
    """blockwise: False (scaled_mm), True (scaled_mm_blockwise) or 2 (the E8M0 GEMM)."""
    return int(lib.fp8q_workspace_bytes(M, N, K, int(blockwise)))


def make_workspace(M: int, N: int, K: int, blockwise, device="cuda") -> torch.Tensor | None:
    """A zero-filled workspace for a GEMM of this shape (None if it needs none)."""
    n = fp8q_workspace_bytes(M, N, K, blockwise)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _ws(ws, M, N, K, blockwise, device):
    """Pointer/size of the caller's workspace; when none is given and the shape
    needs one, a fresh zero-filled buffer (the C ABI itself never allocates)."""
    if ws is None:
        ws = make_workspace(M, N, K, blockwise, device)
    return (ws.data_ptr(), ws.numel() * ws.element_size(), ws) if ws is not None else (None, 0, None)


def fp8q_scaled_mm(a_q: torch.Tensor, b_q: torch.Tensor, a_scale: torch.Tensor,
                   b_scale: torch.Tensor, y=None, workspace=None, stream=None):
    """y [M, N] bf16 = sa * sb * (a_q [M, K] @ b_q [N, K]^T).

    a_scale: fp32 [M] (per token) or [1]; b_scale: fp32 [N] (per channel) or [1].
    """
    for t, n in ((a_q, "a_q"), (b_q, "b_q")):
        _need(t, torch.float8_e4m3fn, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scale, torch.float32, "a_scale")
    _need(b_scale, torch.float32, "b_scale")
    M, K = a_q.shape
    N = b_q.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    if a_scale.numel() not in (1, M) or b_scale.numel() not in (1, N):
        raise ValueError("a_scale must have 1 or M entries, b_scale 1 or N")
    wp, wn, _keep = _ws(workspace, M, N, K, False, a_q.device)
    st = lib.fp8q_scaled_mm(a_q.data_ptr(), b_q.data_ptr(), a_scale.data_ptr(),
                            int(a_scale.numel() == M), b_scale.data_ptr(),
                            int(b_scale.numel() == N), M, N, K, y.data_ptr(), _rowmajor(y, "y"),
                            wp, wn, _stream(stream))
    _check("fp8q_scaled_mm", st)
    return y


def fp8q_scaled_mm_blockwise(a_q: torch.Tensor, b_q: torch.Tensor, a_scale: torch.Tensor,
                             b_scale: torch.Tensor, a_scale_layout: str = "row_major", y=None,
                             workspace=None, stream=None):
    """Block-scaled GEMM: a_scale one fp32 per 1x128 group of A ([M, K/128] row_major or
    [K/128, M] group_major), b_scale fp32 [N/128, K/128]."""
    for t, n in ((a_q, "a_q"), (b_q, "b_q")):
        _need(t, torch.float8_e4m3fn, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scale, torch.float32, "a_scale")
    _need(b_scale, torch.float32, "b_scale")
    M, K = a_q.shape
    N = b_q.shape[0]
    if a_scale_layout == "group_major":
        sm, skb = 1, M
    else:
        sm, skb = K // 128, 1
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    wp, wn, _keep = _ws(workspace, M, N, K, True, a_q.device)
    st = lib.fp8q_scaled_mm_blockwise(a_q.data_ptr(), b_q.data_ptr(), a_scale.data_ptr(), sm, skb,
                                      b_scale.data_ptr(), M, N, K, y.data_ptr(),
                                      _rowmajor(y, "y"), wp, wn, _stream(stream))
    _check("fp8q_scaled_mm_blockwise", st)
    return y


def fp8q_scaled_mm_blockwise_e8m0(a_q: torch.Tensor, b_q: torch.Tensor, a_sf: torch.Tensor,
                                  b_sf: torch.Tensor, a_scale_layout: str = "row_major", y=None,
                                  workspace=None, stream=None):
    """Block-scaled GEMM with E8M0 scale bytes (uint8): a_sf one byte per 1x128 group of
    A ([M, K/128] row_major or [K/128, M] group_major), b_sf [N/128, K/128]; the
    tensor core applies the scales (2^(byte - 127))."""
    for t, n in ((a_q, "a_q"), (b_q, "b_q")):
        _need(t, torch.float8_e4m3fn, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_sf, torch.uint8, "a_sf")
    _need(b_sf, torch.uint8, "b_sf")
    M, K = a_q.shape
    N = b_q.shape[0]
    sm, skb = (1, M) if a_scale_layout == "group_major" else (K // 128, 1)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    wp, wn, _keep = _ws(workspace, M, N, K, 2, a_q.device)
    st = lib.fp8q_scaled_mm_blockwise_e8m0(a_q.data_ptr(), b_q.data_ptr(), a_sf.data_ptr(), sm,
                                           skb, b_sf.data_ptr(), M, N, K, y.data_ptr(),
                                           _rowmajor(y, "y"), wp, wn, _stream(stream))
    _check("fp8q_scaled_mm_blockwise_e8m0", st)
    return y


def interleave_gate_up(t: torch.Tensor, block: int = 128) -> torch.Tensor:
    """Rows of a gate_up tensor [2I, ...] = [gate (I rows) | up (I rows)] reordered
    into 128-row blocks [gate block 0 | up block 0 | gate block 1 | ...], the
    weight layout fp8q_scaled_mm_blockwise_silu_quant reads (a setup-time
    permutation of the weights; use block=1 for their [2I/128, K/128] scales)."""
    n2 = t.shape[0]
    if n2 % (2 * block):
        raise ValueError(f"rows ({n2}) must be a multiple of {2 * block}")
    nb = n2 // (2 * block)
    rest = t.shape[1:]
    g = t[: n2 // 2].reshape(nb, block, *rest)
    u = t[n2 // 2:].reshape(nb, block, *rest)
    return torch.stack([g, u], dim=1).reshape(n2, *rest).contiguous()


def fp8q_scaled_mm_blockwise_silu_quant(a_q: torch.Tensor, b_q: torch.Tensor, a_scale: torch.Tensor,
                                        b_scale: torch.Tensor, a_scale_layout: str = "row_major",
                                        ue8m0=False, q=None, scales=None,
                                        scale_layout: str = "row_major", stream=None):
    """gate_up blockwise GEMM with the SiLU*mul 1x128 quant fused into its epilogue.
    b_q [2I, K] and b_scale [2I/128, K/128] in the interleaved layout of
    interleave_gate_up.  Returns (q e4m3 [M, I], scales [M, I/128] or [I/128, M]).
    Exact mode: bit-identical to fp8q_scaled_mm_blockwise followed by
    fp8q_silu_mul_quant(h, 128); fast mode (default): the same scales, codes
    within the fused-quant tolerance (fp8q_set_fused_quant_exact)."""
    for t, n in ((a_q, "a_q"), (b_q, "b_q")):
        _need(t, torch.float8_e4m3fn, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scale, torch.float32, "a_scale")
    _need(b_scale, torch.float32, "b_scale")
    M, K = a_q.shape
    N2 = b_q.shape[0]
    I = N2 // 2
    sm, skb = (1, M) if a_scale_layout == "group_major" else (K // 128, 1)
    mode = _ue8m0_mode(ue8m0)
    if q is None:
        q = torch.empty((M, I), dtype=torch.float8_e4m3fn, device=a_q.device)
    scales, ssm, ssg = _scales_out(M, I, 128, scale_layout, a_q.device, scales, mode)
    _check("fp8q_scaled_mm_blockwise_silu_quant", lib.fp8q_scaled_mm_blockwise_silu_quant(
        a_q.data_ptr(), b_q.data_ptr(), a_scale.data_ptr(), sm, skb, b_scale.data_ptr(), M, N2, K, mode,
        q.data_ptr(), _rowmajor(q, "q"), scales.data_ptr(), ssm, ssg, _stream(stream)))
    return q, scales


NOALLOC_SCRATCH_BYTES = 16 << 20


def fp8q_scaled_mm_blockwise_noalloc(a_q: torch.Tensor, b_q: torch.Tensor, a_scale: torch.Tensor,
                                     b_scale: torch.Tensor, a_scale_layout: str = "row_major",
                                     y=None, stream=None):
    """fp8q_scaled_mm_blockwise without a workspace: the library's fixed 16 MiB
    scratch array is used instead (calls that overlap on the GPU race)."""
    for t, n in ((a_q, "a_q"), (b_q, "b_q")):
        _need(t, torch.float8_e4m3fn, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scale, torch.float32, "a_scale")
    _need(b_scale, torch.float32, "b_scale")
    M, K = a_q.shape
    N = b_q.shape[0]
    sm, skb = (1, M) if a_scale_layout == "group_major" else (K // 128, 1)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    st = lib.fp8q_scaled_mm_blockwise_noalloc(a_q.data_ptr(), b_q.data_ptr(), a_scale.data_ptr(),
                                              sm, skb, b_scale.data_ptr(), M, N, K, y.data_ptr(),
                                              _rowmajor(y, "y"), _stream(stream))
    _check("fp8q_scaled_mm_blockwise_noalloc", st)
    return y


# --------------------------------------------------------------- fused_qk_norm_rope
def fp8q_qk_norm_rope(qkv: torch.Tensor, num_heads_q: int, num_heads_k: int, num_heads_v: int,
                      head_dim: int, eps: float, q_weight: torch.Tensor, k_weight: torch.Tensor,
                      cos_sin_cache: torch.Tensor, positions: torch.Tensor, is_neox: bool,
                      stream=None) -> torch.Tensor:
    """In place on qkv (bf16 [T, (hq+hk+hv)*D]): per-head RMSNorm of the q and k heads,
    then the rotary embedding at positions (int64 [T]) from cos_sin_cache (fp32
    [max_pos, D] = cos | sin).  Returns qkv."""
    _need(qkv, torch.bfloat16, "qkv")
    _need(q_weight, torch.bfloat16, "q_weight")
    _need(k_weight, torch.bfloat16, "k_weight")
    _need(cos_sin_cache, torch.float32, "cos_sin_cache")
    _need(positions, torch.int64, "positions")
    if not cos_sin_cache.is_contiguous() or not positions.is_contiguous():
        raise ValueError("cos_sin_cache and positions must be contiguous")
    ld = _rowmajor(qkv, "qkv")
    T = qkv.shape[0]
    _check("fp8q_qk_norm_rope", lib.fp8q_qk_norm_rope(
        qkv.data_ptr(), T, ld, num_heads_q, num_heads_k, num_heads_v, head_dim, ctypes.c_float(eps),
        q_weight.data_ptr(), k_weight.data_ptr(), cos_sin_cache.data_ptr(), cos_sin_cache.shape[0],
        positions.data_ptr(), int(bool(is_neox)), _stream(stream)))
    return qkv


# --------------------------------------------------------------- W8A8_INT8
def _quant_i8_out(M, L, group_size, layout, device, q, scales):
    if q is None:
        q = torch.empty((M, L), dtype=torch.int8, device=device)
    elif q.dtype != torch.int8:
        raise TypeError("q must be int8")
    scales, ssm, ssg = _scales_out(M, L, group_size, layout, device, scales)
    return q, scales, ssm, ssg


def fp8q_group_quant_i8(x: torch.Tensor, group_size: int, q=None, scales=None,
                        scale_layout: str = "row_major", stream=None):
    """W8A8_INT8 quant (group_size = K per token, or 128): int8 codes, scale amax/127."""
    _need(x, torch.bfloat16, "x")
    ldx = _rowmajor(x, "x")
    M, K = x.shape
    q, scales, ssm, ssg = _quant_i8_out(M, K, group_size, scale_layout, x.device, q, scales)
    _check("fp8q_group_quant_i8", lib.fp8q_group_quant_i8(
        x.data_ptr(), M, K, ldx, group_size, q.data_ptr(), _rowmajor(q, "q"), scales.data_ptr(), ssm,
        ssg, _stream(stream)))
    return q, scales


def fp8q_rmsnorm_quant_i8(x: torch.Tensor, w: torch.Tensor, eps: float, group_size: int, q=None,
                          scales=None, scale_layout: str = "row_major", stream=None):
    """RMSNorm + W8A8_INT8 quant."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    ldx = _rowmajor(x, "x")
    M, H = x.shape
    q, scales, ssm, ssg = _quant_i8_out(M, H, group_size, scale_layout, x.device, q, scales)
    _check("fp8q_rmsnorm_quant_i8", lib.fp8q_rmsnorm_quant_i8(
        x.data_ptr(), w.data_ptr(), ctypes.c_float(eps), M, H, ldx, group_size, q.data_ptr(),
        _rowmajor(q, "q"), scales.data_ptr(), ssm, ssg, _stream(stream)))
    return q, scales


def fp8q_silu_mul_quant_i8(x: torch.Tensor, group_size: int, q=None, scales=None,
                           scale_layout: str = "row_major", stream=None):
    """SiLU*mul + W8A8_INT8 quant; x [M, 2I] = [gate | up]."""
    _need(x, torch.bfloat16, "x")
    ldx = _rowmajor(x, "x")
    M, I2 = x.shape
    I = I2 // 2
    q, scales, ssm, ssg = _quant_i8_out(M, I, group_size, scale_layout, x.device, q, scales)
    _check("fp8q_silu_mul_quant_i8", lib.fp8q_silu_mul_quant_i8(
        x.data_ptr(), M, I, ldx, group_size, q.data_ptr(), _rowmajor(q, "q"), scales.data_ptr(), ssm,
        ssg, _stream(stream)))
    return q, scales


def fp8q_scaled_mm_i8(a_q: torch.Tensor, b_q: torch.Tensor, a_scale: torch.Tensor,
                      b_scale: torch.Tensor, y=None, workspace=None, stream=None):
    """W8A8_INT8 GEMM: y [M, N] bf16 = sa * sb * (a_q [M, K] @ b_q [N, K]^T), int8 operands,
    exact integer sums; a_scale fp32 [M] or [1], b_scale fp32 [N] or [1]."""
    for t, n in ((a_q, "a_q"), (b_q, "b_q")):
        _need(t, torch.int8, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(a_scale, torch.float32, "a_scale")
    _need(b_scale, torch.float32, "b_scale")
    M, K = a_q.shape
    N = b_q.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    if a_scale.numel() not in (1, M) or b_scale.numel() not in (1, N):
        raise ValueError("a_scale must have 1 or M entries, b_scale 1 or N")
    wp, wn, _keep = _ws(workspace, M, N, K, 3, a_q.device)
    _check("fp8q_scaled_mm_i8", lib.fp8q_scaled_mm_i8(
        a_q.data_ptr(), b_q.data_ptr(), a_scale.data_ptr(), int(a_scale.numel() == M),
        b_scale.data_ptr(), int(b_scale.numel() == N), M, N, K, y.data_ptr(), _rowmajor(y, "y"), wp,
        wn, _stream(stream)))
    return y


# --------------------------------------------------------------- 4-bit microscaled operands
_FP4_FORMATS = {"nvfp4": (0, 16), "mxfp4": (1, 32)}


def _fp4(fmt: str):
    """"nvfp4" / "mxfp4" -> (the ABI's format, values in a group)."""
    try:
        return _FP4_FORMATS[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"format must be 'nvfp4' or 'mxfp4', got {fmt!r}") from None


# the raw current stream of a device, without the Stream object of the public call (3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch_stream(stream, *tensors) -> int | None:
    """The raw stream to launch on; every tensor must be on the current device
    (the kernels, and the outputs allocated for them, go there)."""
    dev = _device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors must be on the current device, cuda:{dev}; one is on {t.device}")
    return _raw_stream(dev) if stream is None else _stream(stream)


def _torch_stream(stream):
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))


def _empty(shape, dtype, like: torch.Tensor, stream):
    """A tensor that belongs to the stream the kernels run on, so that its
    memory is not handed on while they still use it."""
    if stream is None:
        # the cheapest of torch's factories (1.4 us; new_empty 1.9)
        dims = len(shape)
        strides = (shape[1], 1) if dims == 2 else (1,) if dims == 1 else (shape[1] * shape[2], shape[2], 1)
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)
    with torch.cuda.stream(_torch_stream(stream)):
        return torch.empty(shape, dtype=dtype, device=like.device)


_U8, _F32, _I32, _BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16


def _rows(t, dtype, name: str):
    """Rows, columns and row stride of a 2-D CUDA tensor with unit column stride (checked).  A single
    row counts as contiguous, whatever stride it carries."""
    if type(t) is not torch.Tensor or t.dtype is not dtype or not t.is_cuda:
        _need(t, dtype, name)
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        _rowmajor(t, name)                             # raises
    M, K = t.shape
    return M, K, stride[0] if M > 1 else K


def _gscale(t, n: int, name: str):
    if t is None:
        return None
    if type(t) is not torch.Tensor or t.dtype is not _F32 or not t.is_cuda:
        _need(t, _F32, name)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous value(s)")
    return t.data_ptr()


def _sf_shape(rows: int, K: int, group: int):
    return (-(-rows // 128), -(-K // (4 * group)), 512)


def _need_sf(sf, rows: int, K: int, group: int, name: str, lead: int = 1) -> int:
    if type(sf) is not torch.Tensor or sf.dtype is not _U8 or not sf.is_cuda:
        _need(sf, _U8, name)
    n = -(-rows // 128) * -(-K // (4 * group)) * 512 * lead
    if sf.numel() != n or not sf.is_contiguous():
        raise ValueError(f"{name} must be contiguous scale blocks, {lead} x {_sf_shape(rows, K, group)}, "
                         f"got {tuple(sf.shape)}")
    return sf.data_ptr()


def _need_codes(q, name: str, dims: int = 2) -> None:
    if type(q) is not torch.Tensor or q.dtype is not _U8 or not q.is_cuda:
        _need(q, _U8, name)
    if q.dim() != dims or not q.is_contiguous():
        raise ValueError(f"{name} must be contiguous packed codes with {dims} dimensions")


def fp4_sf_shape(rows: int, K: int, fmt: str):
    """Shape of the uint8 scale blocks of a [rows, K] matrix: [ceil(rows / 128),
    ceil(groups / 4), 512]; the scale of row r and group j is byte
    (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4 of block [r // 128, j // 4]."""
    return _sf_shape(rows, K, _fp4(fmt)[1])


def _fp4_quant_out(M, K, group, x, q, sf, stream):
    """Outputs, made here or the caller's (checked): q, its row stride, sf, its address."""
    if q is None:
        q, ldq = _empty((M, K // 2), torch.uint8, x, stream), K // 2
    else:
        _need(q, torch.uint8, "q")
        if tuple(q.shape) != (M, K // 2):
            raise ValueError(f"q must be [{M}, {K // 2}]")
        ldq = _rows(q, _U8, "q")[2]
    if sf is None:
        sf = _empty(_sf_shape(M, K, group), torch.uint8, x, stream)
        return q, ldq, sf, sf.data_ptr()
    return q, ldq, sf, _need_sf(sf, M, K, group, "sf")


def fp8q_fp4_quant(x: torch.Tensor, fmt: str, gscale=None, q=None, sf=None, stream=None):
    """4-bit quantization of bf16 rows [M, K] (K a multiple of 32).  Returns (q uint8 [M, K/2],
    two e2m1 codes a byte; sf uint8 scale blocks of fp4_sf_shape).  fmt "nvfp4": groups of 16,
    e4m3 scales, value = code * scale * gscale (fp32 [1] on the device, or None); "mxfp4": groups
    of 32, E8M0 scales.  Also quantizes weights (a row is an output channel)."""
    M, K, ldx = _rows(x, _BF16, "x")
    f, group = _fp4(fmt)
    g = _gscale(gscale, 1, "gscale")
    q, ldq, sf, sp = _fp4_quant_out(M, K, group, x, q, sf, stream)
    st = lib.fp8q_fp4_quant(x.data_ptr(), M, K, ldx, f, g, q.data_ptr(), ldq, sp,
                            _launch_stream(stream, x, q, sf, gscale))
    _check("fp8q_fp4_quant", st)
    return q, sf


def fp8q_rmsnorm_fp4_quant(x: torch.Tensor, w: torch.Tensor, eps: float, fmt: str, gscale=None, q=None,
                           sf=None, stream=None):
    """RMSNorm + 4-bit quantization; outputs as in fp8q_fp4_quant."""
    M, H, ldx = _rows(x, _BF16, "x")
    if type(w) is not torch.Tensor or w.dtype is not _BF16 or not w.is_cuda:
        _need(w, _BF16, "w")
    f, group = _fp4(fmt)
    if w.numel() != H or not w.is_contiguous():
        raise ValueError(f"w must hold {H} contiguous values")
    g = _gscale(gscale, 1, "gscale")
    q, ldq, sf, sp = _fp4_quant_out(M, H, group, x, q, sf, stream)
    st = lib.fp8q_rmsnorm_fp4_quant(x.data_ptr(), w.data_ptr(), eps, M, H, ldx, f, g, q.data_ptr(), ldq, sp,
                                    _launch_stream(stream, x, w, q, sf, gscale))
    _check("fp8q_rmsnorm_fp4_quant", st)
    return q, sf


def fp8q_silu_mul_fp4_quant(x: torch.Tensor, fmt: str, gscale=None, q=None, sf=None, stream=None):
    """SiLU*mul + 4-bit quantization of x [M, 2I] = [gate | up]; outputs [M, I] as in fp8q_fp4_quant."""
    M, I2, ldx = _rows(x, _BF16, "x")
    f, group = _fp4(fmt)
    if I2 % 2:
        raise ValueError("x must have an even number of columns")
    I = I2 // 2
    g = _gscale(gscale, 1, "gscale")
    q, ldq, sf, sp = _fp4_quant_out(M, I, group, x, q, sf, stream)
    st = lib.fp8q_silu_mul_fp4_quant(x.data_ptr(), M, I, ldx, f, g, q.data_ptr(), ldq, sp,
                                     _launch_stream(stream, x, q, sf, gscale))
    _check("fp8q_silu_mul_fp4_quant", st)
    return q, sf


def fp8q_fp4_dequant(q: torch.Tensor, sf: torch.Tensor, fmt: str, gscale=None, y=None, stream=None):
    """bf16 values [M, K] of packed codes q [M, K/2] and their scale blocks."""
    M, K2, ldq = _rows(q, _U8, "q")
    K = 2 * K2
    f, group = _fp4(fmt)
    sp = _need_sf(sf, M, K, group, "sf")
    g = _gscale(gscale, 1, "gscale")
    y, ldy = _y_out(y, M, K, q, stream)
    st = lib.fp8q_fp4_dequant(q.data_ptr(), ldq, sp, f, g, M, K, y.data_ptr(), ldy,
                                _launch_stream(stream, q, sf, gscale, y))
    _check("fp8q_fp4_dequant", st)
    return y


def _y_out(y, M, N, like, stream):
    """y, made here or the caller's (checked), and its row stride."""
    if y is None:
        return _empty((M, N), torch.bfloat16, like, stream), N
    _need(y, torch.bfloat16, "y")
    if tuple(y.shape) != (M, N):
        raise ValueError(f"y must be [{M}, {N}]")
    return y, _rows(y, _BF16, "y")[2]


def fp8q_scaled_mm_fp4(a_q: torch.Tensor, b_q: torch.Tensor, a_sf: torch.Tensor, b_sf: torch.Tensor, fmt: str,
                       a_gscale=None, b_gscale=None, y=None, stream=None):
    """Block-scaled GEMM on 4-bit operands: y [M, N] bf16 of codes a_q [M, K/2], b_q [N, K/2] and
    their scale blocks (and fp32 [1] tensor scales); N a multiple of 16.  The tensor core applies
    the scales."""
    _need_codes(a_q, "a_q")
    _need_codes(b_q, "b_q")
    f, group = _fp4(fmt)
    (M, K2), N = a_q.shape, b_q.shape[0]
    if b_q.shape[1] != K2:
        raise ValueError("a_q and b_q must have the same depth")
    ap = _need_sf(a_sf, M, 2 * K2, group, "a_sf")
    bp = _need_sf(b_sf, N, 2 * K2, group, "b_sf")
    ga, gb = _gscale(a_gscale, 1, "a_gscale"), _gscale(b_gscale, 1, "b_gscale")
    y, ldy = _y_out(y, M, N, a_q, stream)
    st = lib.fp8q_scaled_mm_fp4(a_q.data_ptr(), b_q.data_ptr(), ap, bp, f, ga, gb, M, N, 2 * K2, y.data_ptr(), ldy,
                                _launch_stream(stream, a_q, b_q, a_sf, b_sf, a_gscale, b_gscale, y))
    _check("fp8q_scaled_mm_fp4", st)
    return y


# --------------------------------------------------------------- experts
_SCORING = {"softmax": 0, "sigmoid": 1}


def fp8q_moe_route(logits: torch.Tensor, top_k: int, scoring: str = "softmax", bias=None, num_groups: int = 1,
                   topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, weights=None, ids=None,
                   stream=None):
    """Experts of each token from router logits [T, E] (fp32 or bf16).  Scores are a softmax over
    the experts or a sigmoid of each; `bias` (fp32 [E]) is added for the selection only; with
    topk_groups < num_groups only experts of the best groups of neighbours are selected (a group
    counts with its largest key, with a bias the sum of its two largest).  Equal keys go to the
    lowest index; -inf or NaN logits mask.  Returns (weights fp32 [T, top_k], ids int32 [T, top_k])
    in descending order of the key; weights are scores, divided by their sum if `renormalize`,
    times `scale`."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if top_k <= 0:
        raise ValueError("top_k must be positive")
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
    ld = _rowmajor(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _gscale(bias, E, "bias")
    if weights is None:
        weights = _empty((T, top_k), torch.float32, logits, stream)
    else:
        _need_entries(weights, torch.float32, T, top_k, "weights")
    if ids is None:
        ids = _empty((T, top_k), torch.int32, logits, stream)
    else:
        _need_entries(ids, torch.int32, T, top_k, "ids")
    st = lib.fp8q_moe_route(logits.data_ptr(), logits.dtype is torch.bfloat16, T, E, ld if T > 1 else max(ld, E),
                            top_k, _SCORING[scoring], None if bias is None else bias.data_ptr(), num_groups,
                            topk_groups, bool(renormalize), scale, weights.data_ptr(), ids.data_ptr(),
                            _launch_stream(stream, logits, bias, weights, ids))
    _check("fp8q_moe_route", st)
    return weights, ids


def _need_entries(t, dtype, T, k, name):
    if type(t) is not torch.Tensor or t.dtype is not dtype or not t.is_cuda:
        _need(t, dtype, name)
    if t.shape != (T, k) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{T}, {k}]")


class MoePlan(NamedTuple):
    """What fp8q_moe_plan returns: int32 tensors."""
    offsets: torch.Tensor      # [E + 1] first row of each expert
    sf_offsets: torch.Tensor   # [E + 1] first block row of each expert's scales
    pos: torch.Tensor          # [T, top_k] an entry's row, or -1
    sf_row: torch.Tensor       # [T, top_k] the row whose place its scales take, or -1


def fp8q_moe_plan(ids: torch.Tensor, num_experts: int, stream=None) -> MoePlan:
    """Rows of the (token, slot) entries of ids int32 [T, top_k], ordered by expert, in entry order
    within an expert; ids outside [0, num_experts) get none."""
    _need(ids, torch.int32, "ids")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be contiguous [T, top_k]")
    if num_experts <= 0:
        raise ValueError("num_experts must be positive")
    n = ids.numel()
    offsets, sf_offsets = (_empty((num_experts + 1,), torch.int32, ids, stream) for _ in range(2))
    pos, sf_row = (_empty(ids.shape, torch.int32, ids, stream) for _ in range(2))
    nws = lib.fp8q_moe_plan_workspace_bytes(n, num_experts)
    ws = _empty((nws,), torch.uint8, ids, stream) if nws else None
    st = lib.fp8q_moe_plan(ids.data_ptr(), n, num_experts, offsets.data_ptr(), sf_offsets.data_ptr(),
                           pos.data_ptr(), sf_row.data_ptr(), None if ws is None else ws.data_ptr(), nws,
                           _launch_stream(stream, ids))
    _check("fp8q_moe_plan", st)
    return MoePlan(offsets, sf_offsets, pos, sf_row)


def moe_sf_rows(n: int, num_experts: int) -> int:
    """Rows of scale blocks that n rows of the experts may take: every expert's begin a block row."""
    return 128 * (n // 128 + min(n, num_experts))


def fp8q_moe_fp4_quant(x: torch.Tensor, plan: MoePlan, fmt: str, gscale=None, stream=None):
    """fp8q_fp4_quant of tokens [T, H], each written to the rows of its experts.  Returns
    (q [T * top_k, H/2], sf) as fp8q_grouped_mm_fp4 reads them."""
    T, K, ldx = _rows(x, _BF16, "x")
    f, group = _fp4(fmt)
    _need_entries(plan.pos, torch.int32, T, plan.pos.shape[1], "plan.pos")
    _need_entries(plan.sf_row, torch.int32, T, plan.pos.shape[1], "plan.sf_row")
    n = plan.pos.numel()
    g = _gscale(gscale, 1, "gscale")
    q = _empty((n, K // 2), torch.uint8, x, stream)
    sf = _empty(_sf_shape(moe_sf_rows(n, plan.offsets.numel() - 1), K, group), torch.uint8, x, stream)
    st = lib.fp8q_moe_fp4_quant(x.data_ptr(), T, K, ldx, plan.pos.shape[1], plan.pos.data_ptr(),
                                plan.sf_row.data_ptr(), f, g, q.data_ptr(), K // 2, sf.data_ptr(),
                                _launch_stream(stream, x, gscale, *plan))
    _check("fp8q_moe_fp4_quant", st)
    return q, sf


def _grouped(a_q, b_q, a_sf, b_sf, fmt, plan, a_gscale, b_gscale):
    _need_codes(a_q, "a_q")
    _need_codes(b_q, "b_q", 3)
    f, group = _fp4(fmt)
    (M, K2), (E, N, Kb) = a_q.shape, b_q.shape
    if Kb != K2:
        raise ValueError("a_q and b_q must have the same depth")
    for t, name in ((plan.offsets, "plan.offsets"), (plan.sf_offsets, "plan.sf_offsets")):
        _need(t, torch.int32, name)
        if t.numel() != E + 1 or not t.is_contiguous():
            raise ValueError(f"{name} must hold {E + 1} contiguous values")
    if plan.pos.numel() != M:
        raise ValueError(f"a_q has {M} rows, the plan {plan.pos.numel()} entries")
    _need_sf(a_sf, moe_sf_rows(M, E), 2 * K2, group, "a_sf")
    _need_sf(b_sf, N, 2 * K2, group, "b_sf", E)
    return f, group, M, N, 2 * K2, E, _gscale(a_gscale, 1, "a_gscale"), _gscale(b_gscale, E, "b_gscale")


def fp8q_grouped_mm_fp4(a_q: torch.Tensor, b_q: torch.Tensor, a_sf: torch.Tensor, b_sf: torch.Tensor, fmt: str,
                        plan: MoePlan, a_gscale=None, b_gscale=None, y=None, stream=None):
    """Each expert's rows times its weights: y [M, N] bf16 from a_q [M, K/2] and a_sf (rows as the
    plan orders them), b_q [E, N, K/2] and b_sf [E, *fp4_sf_shape(N, K, fmt)]; a_gscale fp32 [1],
    b_gscale fp32 [E].  Rows without an expert are not written."""
    f, group, M, N, K, E, ga, gb = _grouped(a_q, b_q, a_sf, b_sf, fmt, plan, a_gscale, b_gscale)
    y, ldy = _y_out(y, M, N, a_q, stream)
    st = lib.fp8q_grouped_mm_fp4(a_q.data_ptr(), b_q.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(), f, ga, gb,
                                 plan.offsets.data_ptr(), plan.sf_offsets.data_ptr(), E, M, N, K, y.data_ptr(), ldy,
                                 _launch_stream(stream, a_q, b_q, a_sf, b_sf, a_gscale, b_gscale, y, *plan))
    _check("fp8q_grouped_mm_fp4", st)
    return y


def fp8q_grouped_mm_fp4_silu_quant(a_q: torch.Tensor, b_q: torch.Tensor, a_sf: torch.Tensor, b_sf: torch.Tensor,
                                   fmt: str, plan: MoePlan, a_gscale=None, b_gscale=None, gscale=None, stream=None):
    """The experts' gate_up product with SiLU*mul and the next quantization in its epilogue: b_q
    [E, 2I, K/2] = [gate | up] rows, I a multiple of 128.  Returns (q [M, I/2], sf) at the plan's
    rows, with tensor scale `gscale`."""
    f, group, M, N, K, E, ga, gb = _grouped(a_q, b_q, a_sf, b_sf, fmt, plan, a_gscale, b_gscale)
    if N % 2:
        raise ValueError(f"b_q must have as many up rows as gate rows, got {N} in all")
    g = _gscale(gscale, 1, "gscale")
    I = N // 2
    q = _empty((M, I // 2), torch.uint8, a_q, stream)
    sf = _empty(_sf_shape(moe_sf_rows(M, E), I, group), torch.uint8, a_q, stream)
    st = lib.fp8q_grouped_mm_fp4_silu_quant(
        a_q.data_ptr(), b_q.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(), f, ga, gb, plan.offsets.data_ptr(),
        plan.sf_offsets.data_ptr(), E, M, I, K, g, q.data_ptr(), sf.data_ptr(),
        _launch_stream(stream, a_q, b_q, a_sf, b_sf, a_gscale, b_gscale, gscale, *plan))
    _check("fp8q_grouped_mm_fp4_silu_quant", st)
    return q, sf


def fp8q_moe_combine(o: torch.Tensor, plan: MoePlan, weights: torch.Tensor, y=None, stream=None):
    """y [T, H] bf16 = the sum over slots of weights [T, top_k] times rows plan.pos of o (bf16)."""
    n, H, ldo = _rows(o, _BF16, "o")
    T, k = plan.pos.shape
    _need_entries(plan.pos, torch.int32, T, k, "plan.pos")
    _need_entries(weights, torch.float32, T, k, "weights")
    if n != T * k:
        raise ValueError(f"o must have {T * k} rows")
    y, ldy = _y_out(y, T, H, o, stream)
    st = lib.fp8q_moe_combine(o.data_ptr(), ldo, plan.pos.data_ptr(), weights.data_ptr(), T, k, H,
                              y.data_ptr(), ldy, _launch_stream(stream, o, weights, y, plan.pos))
    _check("fp8q_moe_combine", st)
    return y


def make_moe_workspace(T: int, top_k: int, num_experts: int, H: int, I: int, fmt: str, device="cuda"):
    """A workspace for fp8q_moe_experts_fp4 of up to T tokens (any content)."""
    n = lib.fp8q_moe_experts_fp4_workspace_bytes(T, top_k, num_experts, H, I, _fp4(fmt)[0])
    return torch.empty(n, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=1024)
def _experts_bytes(T, k, E, H, I, f) -> int:
    return lib.fp8q_moe_experts_fp4_workspace_bytes(T, k, E, H, I, f)


def fp8q_moe_experts_fp4(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor,
                         w13_sf: torch.Tensor, w2: torch.Tensor, w2_sf: torch.Tensor, fmt: str, x_gscale=None,
                         w13_gscale=None, h_gscale=None, w2_gscale=None, y=None, workspace=None, stream=None):
    """The experts' pass over tokens x bf16 [T, H]: y[t] = sum_j weights[t, j] W2_e quant(silu(gate) up),
    e = ids[t, j].  w13 codes [E, 2I, H/2] = [gate | up], w2 codes [E, H, I/2], with scale blocks
    [E, *fp4_sf_shape(rows, cols, fmt)]; x_gscale, h_gscale fp32 [1], w13_gscale, w2_gscale fp32 [E].
    Four launches for up to 128 (token, slot) entries, five to seven for more; ids outside [0, E) add
    nothing."""
    T, H, ldx = _rows(x, _BF16, "x")
    _need_codes(w13, "w13", 3)
    _need_codes(w2, "w2", 3)
    f, group = _fp4(fmt)
    E, I2, Hh = w13.shape
    I = I2 // 2
    if Hh * 2 != H or I2 % 2 or w2.shape != (E, H, I // 2):
        raise ValueError(f"x {tuple(x.shape)}, w13 {tuple(w13.shape)} and w2 {tuple(w2.shape)} do not fit")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise TypeError("ids must be a 2-D CUDA tensor")
    k = ids.shape[1]
    _need_entries(ids, torch.int32, T, k, "ids")
    _need_entries(weights, torch.float32, T, k, "weights")
    s13, s2 = _need_sf(w13_sf, I2, H, group, "w13_sf", E), _need_sf(w2_sf, H, I, group, "w2_sf", E)
    gx, gh = _gscale(x_gscale, 1, "x_gscale"), _gscale(h_gscale, 1, "h_gscale")
    g13, g2 = _gscale(w13_gscale, E, "w13_gscale"), _gscale(w2_gscale, E, "w2_gscale")
    y, ldy = _y_out(y, T, H, x, stream)
    if workspace is None:
        workspace = _empty((_experts_bytes(T, k, E, H, I, f),), _U8, x, stream)
    else:
        _need(workspace, torch.uint8, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    st = lib.fp8q_moe_experts_fp4(
        x.data_ptr(), T, ldx, ids.data_ptr(), weights.data_ptr(), k, E, H, I, f, w13.data_ptr(), s13, w2.data_ptr(),
        s2, gx, g13, gh, g2, y.data_ptr(), ldy, workspace.data_ptr(), workspace.numel(),
        _launch_stream(stream, x, ids, weights, w13, w13_sf, w2, w2_sf, x_gscale, w13_gscale, h_gscale, w2_gscale, y,
                       workspace))
    _check("fp8q_moe_experts_fp4", st)
    return y


def fp8q_fp4_sf_bytes(rows: int, K: int, fmt: str) -> int:
    return int(lib.fp8q_fp4_sf_bytes(rows, K, _fp4(fmt)[0]))


def fp8q_moe_plan_workspace_bytes(n: int, num_experts: int) -> int:
    return int(lib.fp8q_moe_plan_workspace_bytes(n, num_experts))


def fp8q_moe_experts_fp4_workspace_bytes(T: int, top_k: int, num_experts: int, H: int, I: int, fmt: str) -> int:
    return int(lib.fp8q_moe_experts_fp4_workspace_bytes(T, top_k, num_experts, H, I, _fp4(fmt)[0]))


def fp8q_select_gemm_variant(M: int, N: int, K: int, blockwise: bool) -> dict:
    v = GemmVariant()
    _check("fp8q_select_gemm_variant", lib.fp8q_select_gemm_variant(M, N, K, int(blockwise),
                                                                    ctypes.byref(v)))
    return v.as_dict()


def fp8q_force_gemm_variant(swap_ab: int | None = None, split_k: int = 1, block_n: int = 128,
                            cta_pair: int = 0):
    """Force a GEMM variant for the following calls (testing/tuning); no args = automatic."""
    if swap_ab is None:
        _check("fp8q_force_gemm_variant", lib.fp8q_force_gemm_variant(None))
        return
    v = GemmVariant(int(swap_ab), int(split_k), int(block_n), int(cta_pair))
    _check("fp8q_force_gemm_variant", lib.fp8q_force_gemm_variant(ctypes.byref(v)))


def fp8q_set_fused_quant_exact(exact: bool) -> None:
    """Arithmetic of the producer-fused quant ops for the calls that follow
    (process-wide): False (default) = fast y within the fused tolerance with
    exact scales, True = bit-exact codes and scales."""
    _check("fp8q_set_fused_quant_exact", lib.fp8q_set_fused_quant_exact(1 if exact else 0))


def fp8q_get_fused_quant_exact() -> bool:
    return bool(lib.fp8q_get_fused_quant_exact())


def fp8q_last_device_status(stream=None) -> int:
    return int(lib.fp8q_last_device_status(_stream(stream)))


def fp8q_status_string(status: int) -> str:
    return lib.fp8q_status_string(status).decode()


def fp8q_version() -> str:
    return lib.fp8q_version().decode()
