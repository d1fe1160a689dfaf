"""Oracle of the 4-bit microscaled operators and of routing to experts -- TEST
INFRASTRUCTURE ONLY, written from the definitions in include/fp8q_fp4.h, in
numpy fp64 except where a definition fixes fp32.  Shares nothing with the CUDA
sources.

Values are fp64 arrays; codes are uint8, one 4-bit code per byte ("unpacked")
or two ("packed", the lower index in the low half); scales are kept as their
stored bytes [rows, groups] and laid out in 128 x 4 blocks by `store_scales`.
"""
from __future__ import annotations

import numpy as np

GROUP = {"nvfp4": 16, "mxfp4": 32}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f32(v):
    with np.errstate(over="ignore"):
        return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def bf16(v):
    """fp64 -> nearest bf16 value (ties to even, one rounding), as fp64."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(v), np.rint(v / step) * step, v)


def e2m1_encode(v):
    """Codes 0..15: nearest, ties to the even code, saturating; the sign kept."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 6.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))   # of the binade; ties to even multiples
    r = np.rint(a / step) * step                              # 2 and 4 close their binades from below
    return (np.searchsorted(GRID, r) + 8 * np.signbit(v)).astype(np.uint8)


def e2m1_decode(c):
    c = np.asarray(c)
    return np.where(c & 8, -1.0, 1.0) * GRID[c & 7]


def e4m3_encode(v):
    """Non-negative values -> e4m3 bytes, nearest, ties to even, saturating at 448."""
    v = np.minimum(np.asarray(v, np.float64), 448.0)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    r = np.rint(v / step) * step
    m, e = np.frexp(r)                                        # r = m 2^e, 1/2 <= m < 1
    normal = (e + 6) * 8 + np.rint(m * 16 - 8)
    return np.where(r < 2.0 ** -6, np.rint(r * 512), normal).astype(np.uint8)


def e4m3_decode(b):
    b = np.asarray(b).astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.ldexp(1.0, e - 10))


def scale_values(b, fmt):
    return e4m3_decode(b) if fmt == "nvfp4" else np.ldexp(1.0, np.asarray(b).astype(np.int64) - 127)


def quantize(y, fmt, g=1.0):
    """y [M, K] -> (unpacked codes [M, K], scale bytes [M, K / group])."""
    y = np.asarray(y, np.float64)
    M, K = y.shape
    y3 = y.reshape(M, -1, GROUP[fmt])
    amax = np.abs(y3).max(axis=2)
    if fmt == "nvfp4":
        b = e4m3_encode(f32(f32(amax / 6) / g))
        d = f32(e4m3_decode(b) * g)[:, :, None]
    else:
        u = f32(np.maximum(amax, float(np.float32(1e-10))) / 6)
        m, e = np.frexp(u)
        b = np.where(np.isinf(u), 254, np.minimum(np.where(m == 0.5, e - 1, e) + 127, 254)).astype(np.uint8)
        d = scale_values(b, fmt)[:, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(d > 0, f32(y3 / d), 0 * y3)
    t = np.where(np.isnan(t), np.copysign(6.0, y3), t)        # inf / d stays inf; inf / inf cannot occur
    return e2m1_encode(np.copysign(t, y3)).reshape(M, K), b


def values(codes, b, fmt, g=1.0):
    """Unpacked codes and scale bytes -> fp64 values."""
    return e2m1_decode(codes) * np.repeat(scale_values(b, fmt), GROUP[fmt], axis=-1) * g


def dequant_bf16(codes, b, fmt, g=1.0):
    t = e2m1_decode(codes) * np.repeat(scale_values(b, fmt), GROUP[fmt], axis=-1)
    return bf16(f32(f32(t) * g))


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(q):
    out = np.empty((*q.shape[:-1], 2 * q.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = q & 15, q >> 4
    return out


def _place(rows, groups):
    r, j = np.arange(rows)[:, None], np.arange(groups)[None, :]
    kb = -(-groups // 4)
    return (r // 128 * kb + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4


def store_scales(b, fill=0):
    """Scale bytes [rows, groups] -> blocks [ceil(rows / 128), ceil(groups / 4), 512]."""
    rows, groups = b.shape
    rb, kb = -(-rows // 128), -(-groups // 4)
    out = np.full(rb * kb * 512, fill, np.uint8)
    out[_place(rows, 4 * kb)] = 0
    out[_place(rows, groups)] = b
    return out.reshape(rb, kb, 512)


def load_scales(blocks, rows, groups):
    return blocks.reshape(-1)[_place(rows, groups)]


def rmsnorm(x, w, eps):
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x * x).sum(axis=1, keepdims=True) / x.shape[1] + float(np.float32(eps)))
    return bf16(bf16(x * r) * w)


def silu_mul(gate, up):
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up


def route(logits, k, scoring, bias=None, groups=1, topg=1, renorm=True, scale=1.0):
    """(weights fp64 [T, k], ids [T, k]) of logits fp64 [T, E]."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64)) + 0.0
    T, E = l.shape
    W, I = np.zeros((T, k)), np.zeros((T, k), np.int32)
    for t in range(T):
        x = l[t]
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1 / (1 + np.exp(-x))
        else:
            z = np.array([0.0 if v == -np.inf else 1.0 if v == x.max() else np.exp(v - x.max()) for v in x])
            s = z / z.sum() if z.sum() > 0 else z
        key = x if bias is None else np.where(x == -np.inf, -np.inf, s + bias)
        allowed = list(range(E))
        if topg < groups:
            size = E // groups
            best = []
            for g in range(groups):
                top = sorted(key[g * size:(g + 1) * size], reverse=True)[:1 if bias is None else 2]
                best.append(sum(top))
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:topg]
            allowed = [e for e in allowed if e // size in kept]
        ids = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        w = s[ids]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        W[t], I[t] = w * scale, ids
    return W, I


def plan(ids, E):
    """(offsets, sf_offsets, pos, sf_row) of ids [T, k]."""
    flat = ids.reshape(-1)
    pos, row = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    off, sf = [0], [0]
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        pos[at] = off[-1] + np.arange(at.size)
        row[at] = 128 * sf[-1] + np.arange(at.size)
        off.append(off[-1] + at.size)
        sf.append(sf[-1] + -(-at.size // 128))
    return np.array(off, np.int32), np.array(sf, np.int32), pos.reshape(ids.shape), row.reshape(ids.shape)
