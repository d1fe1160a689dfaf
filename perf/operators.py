"""Cases for the 4-bit microscaled path: quantisation, its block-scaled product, routing to experts and
the experts' products.

Formats.  A value is held as code * sf * g: `code` a 4-bit e2m1 number (0, .5, 1, 1.5, 2, 3, 4, 6 and
their negatives, two to a byte, the lower index in the low half), `sf` one scale for a group of
consecutive values of a row, `g` one fp32 scale of the tensor (or of the expert), 1 where there is none.
  nvfp4  groups of 16, sf an e4m3 number:   sf = e4m3(min((amax / 6) / g, 448)), code = e2m1(y / (sf g))
  mxfp4  groups of 32, sf a power of two:   sf = 2^ceil(log2(max(amax, 1e-10) / 6)), code = e2m1(y / sf)
Scale bytes are stored in blocks of 128 rows x 4 groups: [ceil(rows / 128), ceil(groups / 4), 512], the
byte of row r and group j at (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4 of block (r // 128, j // 4);
bytes of absent rows and groups are zero in weights.

Every rounding that decides a code is part of the operator's definition: y is rounded to bf16 once
(RMSNorm: twice, bf16(bf16(x r) w)), each quotient and the product sf g to fp32, codes and e4m3 scales
to the nearest, ties to even.  Between the experts' two products nothing is rounded but to the codes.
"""
import math

import torch

own = False
GROUP = {"nvfp4": 16, "mxfp4": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decode step entering a linear layer of hidden size 4096
        {"name": "quant rmsnorm 1 token", "op": "quant", "kind": "rmsnorm", "fmt": "nvfp4", "m": 1, "k": 4096, "pad": 0, "gscale": False},
        # an attention output of 1000 tokens, read out of wider rows
        {"name": "quant plain 1000 of wider rows", "op": "quant", "kind": "plain", "fmt": "mxfp4", "m": 1000, "k": 5120, "pad": 1024, "gscale": False},
        # a prefill chunk between gate_up and down of an MLP with 12288 channels
        {"name": "quant silu 8192", "op": "quant", "kind": "silu", "fmt": "nvfp4", "m": 8192, "k": 12288, "pad": 0, "gscale": True},
        # decode: one token through a gate_up layer, bound by reading the weights
        {"name": "mm 1 x 51200 x 5120", "op": "mm", "fmt": "nvfp4", "m": 1, "n": 51200, "k": 5120, "gscale": True},
        # decode: a batch of 16 through a down layer
        {"name": "mm 16 x 4096 x 12288", "op": "mm", "fmt": "mxfp4", "m": 16, "n": 4096, "k": 12288, "gscale": False},
        # a ragged chunk of a prompt through a gate_up layer
        {"name": "mm 1000 x 24576 x 4096", "op": "mm", "fmt": "mxfp4", "m": 1000, "n": 24576, "k": 4096, "gscale": False},
        # prefill: the widest layer of the benchmark's linear stack
        {"name": "mm 8192 x 51200 x 5120", "op": "mm", "fmt": "nvfp4", "m": 8192, "n": 51200, "k": 5120, "gscale": True},
        # the router of one decoded token
        {"name": "route 1 of 128", "op": "route", "scoring": "softmax", "t": 1, "e": 128, "k": 8, "groups": 1, "topg": 1, "bias": False, "renorm": True, "bf16": True},
        # the router of a prefill chunk: balanced by a bias, groups limited
        {"name": "route 8192 of 256 grouped", "op": "route", "scoring": "sigmoid", "t": 8192, "e": 256, "k": 8, "groups": 8, "topg": 4, "bias": True, "renorm": True, "bf16": False},
        # the experts of one decoded token
        {"name": "experts 1 token 8 of 128", "op": "experts", "fmt": "nvfp4", "t": 1, "e": 128, "k": 8, "h": 2048, "i": 768, "gscale": True},
        # a ragged mid-size batch, experts of uneven load
        {"name": "experts 333 tokens 6 of 64", "op": "experts", "fmt": "mxfp4", "t": 333, "e": 64, "k": 6, "h": 2048, "i": 1408, "gscale": False},
        # a prefill chunk
        {"name": "experts 4096 tokens 8 of 128", "op": "experts", "fmt": "nvfp4", "t": 4096, "e": 128, "k": 8, "h": 2048, "i": 768, "gscale": True},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("quant", "mm", "mm", "route", "experts", "experts"))
    fmt = rng.choice(("nvfp4", "mxfp4"))
    gscale = fmt == "nvfp4" and rng.random() < 0.5
    if op == "quant":
        kind = rng.choice(("plain", "rmsnorm", "silu"))
        k = _log(rng, 512, 16384, 32)
        m = _log(rng, 1, min(8192, 8192 * 12288 // k))
        return {"op": op, "kind": kind, "fmt": fmt, "m": m, "k": k, "pad": rng.choice((0, 64, 1000)), "gscale": gscale}
    if op == "mm":
        n, k = _log(rng, 512, 51200, 16), _log(rng, 512, 25600, 32)
        m = _log(rng, 1, max(1, min(8192, 8192 * 51200 * 5120 // (n * k))))
        return {"op": op, "fmt": fmt, "m": m, "n": n, "k": k, "gscale": gscale}
    if op == "route":
        groups = rng.choice((1, 4, 8))
        e = _log(rng, 16, 512 // groups, 8) * groups if groups > 1 else _log(rng, 16, 512, 1)
        topg = rng.randint(max(1, groups // 4), groups)
        k = rng.randint(1, min(16, e // groups * topg))
        return {"op": op, "scoring": rng.choice(("softmax", "sigmoid")), "t": _log(rng, 1, 8192), "e": e, "k": k, "groups": groups, "topg": topg,
                "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7, "bf16": rng.random() < 0.5}
    e = rng.choice((8, 16, 32, 64, 128))
    h, i = _log(rng, 512, 2048, 64), _log(rng, 256, 768, 128)
    k = rng.randint(1, min(8, e))
    return {"op": op, "fmt": fmt, "t": _log(rng, 1, 4096), "e": e, "k": k, "h": h, "i": i, "gscale": gscale}


# ------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, cols):
    """Heavy-tailed values with a few large channels, as in the residual stream, in bf16."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x.div_(torch.rand(rows, 1, device="cuda", generator=g).clamp_(0.05).sqrt_())
    big = torch.randint(0, cols, (max(1, cols // 100),), device="cuda", generator=g)
    x[:, big] *= 20.0
    return x.to(torch.bfloat16)


def _weights(g, rows, cols, fmt, gs):
    """Codes and stored scale bytes of a weight ~ N(0, 0.02) [rows, cols]."""
    w = (torch.randn(rows, cols, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
    code, sf = _quantise(w.float(), fmt, gs)
    return _pack(code), _store_scales(sf, fmt)


def prepare(case, seed):
    g, s = _gen(seed), {"case": dict(case)}
    op = case["op"]
    one = lambda v: torch.tensor([v], device="cuda", dtype=torch.float32)  # noqa: E731
    if op == "quant":
        wide = case["k"] * (2 if case["kind"] == "silu" else 1)
        x = _activations(g, case["m"], wide + case["pad"])
        s["x"] = x[:, :wide]
        if case["kind"] == "rmsnorm":
            s["w"] = (1 + 0.1 * torch.randn(case["k"], device="cuda", generator=g)).to(torch.bfloat16)
        s["gs"] = one(0.037) if case["gscale"] else None
    elif op == "mm":
        s["ags"], s["bgs"] = (one(0.031), one(0.00007)) if case["gscale"] else (None, None)
        x = _activations(g, case["m"], case["k"])
        code, sf = _quantise(x.float(), case["fmt"], s["ags"])
        s["a"], s["asf"] = _pack(code), _store_scales(sf, case["fmt"])
        s["b"], s["bsf"] = _weights(g, case["n"], case["k"], case["fmt"], s["bgs"])
    elif op == "route":
        t, e = case["t"], case["e"]
        l = 1.5 * torch.randn(t, e, device="cuda", generator=g) + torch.randn(e, device="cuda", generator=g)
        s["logits"] = l.to(torch.bfloat16) if case["bf16"] else l
        s["bias"] = 0.2 * torch.randn(e, device="cuda", generator=g) if case["bias"] else None
    else:
        t, e, k, h, i = (case[n] for n in ("t", "e", "k", "h", "i"))
        gen = torch.rand(e, device="cuda", generator=g) * 0.0004 + 0.0001
        s["g13"], s["g2"] = (gen, gen.flip(0).contiguous()) if case["gscale"] else (None, None)
        s["gx"], s["gh"] = (one(0.02), one(0.004)) if case["gscale"] else (None, None)
        rep = lambda v, n: None if v is None else v.repeat_interleave(n).view(-1, 1)  # noqa: E731
        blocks = lambda n: -(-n // 128) * 128  # noqa: E731
        s["w13"], s["w2"] = (torch.empty(e, n, c // 2, device="cuda", dtype=torch.uint8) for n, c in ((2 * i, h), (h, i)))
        gr = GROUP[case["fmt"]]
        s["w13_sf"], s["w2_sf"] = (torch.empty(e, blocks(n) // 128, -(-(c // gr) // 4), 512, device="cuda", dtype=torch.uint8) for n, c in ((2 * i, h), (h, i)))
        for j in range(e):  # one expert at a time: the largest case has 600 million weights
            s["w13"][j], s["w13_sf"][j] = _weights(g, 2 * i, h, case["fmt"], None if s["g13"] is None else s["g13"][j:j + 1])
            s["w2"][j], s["w2_sf"][j] = _weights(g, h, i, case["fmt"], None if s["g2"] is None else s["g2"][j:j + 1])
        s["x"] = torch.randn(t, h, device="cuda", generator=g).to(torch.bfloat16)
        l = torch.randn(t, e, device="cuda", generator=g) + 0.5 * torch.randn(e, device="cuda", generator=g)
        w, ids = torch.topk(torch.softmax(l, 1), k, dim=1)
        s["weights"], s["ids"] = (w / w.sum(1, keepdim=True)).contiguous(), ids.to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------------------- the operators, plainly
def _code(v):
    """e2m1 codes 0..15 of v: nearest, ties to the even code, saturating at 6."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5
    return c + 8 * torch.signbit(v).to(torch.uint8)


def _quantise(y, fmt, gs):
    """Codes [M, K] (one a byte) and scales [M, groups] in fp32 of y (fp32, holding bf16 values)."""
    m, k = y.shape
    amax = y.view(m, -1, GROUP[fmt]).abs().amax(2)
    if fmt == "nvfp4":
        u = (amax.double() / 6).float()
        u = u if gs is None else (u.double() / gs.double()).float()
        sf = u.clamp(max=448.0).to(torch.float8_e4m3fn).float()
        d = sf if gs is None else sf * gs
    else:
        u = (amax.clamp(min=1e-10).double() / 6).float()
        frac, exp = torch.frexp(u)  # u = frac 2^exp, 1/2 <= frac < 1
        d = sf = torch.ldexp(torch.ones_like(u), exp - (frac == 0.5).to(exp.dtype))
    d = d.repeat_interleave(GROUP[fmt], 1)
    return _code(torch.where(d > 0, y / d, y * 0)), sf


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(q):
    """Packed codes [..., K / 2] -> their values [..., K] in fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    return table[torch.stack((q & 15, q >> 4), -1).int()].flatten(-2)


def _store_scales(sf, fmt):
    """Scales [rows, groups] -> bytes in 128 x 4 blocks."""
    rows, groups = sf.shape
    b = sf.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "nvfp4" else (torch.frexp(sf)[1] + 126).to(torch.uint8)
    b = torch.nn.functional.pad(b, (0, -groups % 4, 0, -rows % 128))
    return b.view(-1, 4, 32, b.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, b.shape[1] // 4, 512).contiguous()


def _load_scales(b, rows, groups, fmt):
    """Bytes [..., row blocks, group blocks, 512] -> scales [..., rows, groups] in fp32."""
    lead = b.shape[:-3]
    v = b.reshape(-1, b.shape[-3], b.shape[-2], 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(*lead, b.shape[-3] * 128, -1)[..., :rows, :groups].contiguous()
    return v.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.ldexp(torch.ones((), device=b.device), v.int() - 127)


def _values(q, sf, fmt):
    """Packed codes [..., rows, K / 2] and stored scales -> code * sf in fp32."""
    v = _unpack(q)
    s = _load_scales(sf, v.shape[-2], v.shape[-1] // GROUP[fmt], fmt)
    return v.unflatten(-1, (-1, GROUP[fmt])).mul_(s.unsqueeze(-1)).flatten(-2)


def _silu_mul(h):
    """bf16(silu(gate) up) of rows [gate | up], as fp32: in 64 bits, since a value next to a rounding border decides a code."""
    gate, up = h.double().chunk(2, -1)
    return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16).float()


def _quant(s):
    c = s["case"]
    x = s["x"].float()
    if c["kind"] == "rmsnorm":
        r = 1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-6)
        x = ((x.double() * r).to(torch.bfloat16).float() * s["w"].float()).to(torch.bfloat16).float()
    elif c["kind"] == "silu":
        x = _silu_mul(x)
    code, sf = _quantise(x, c["fmt"], s["gs"])
    v = _values(_pack(code), _store_scales(sf, c["fmt"]), c["fmt"])
    return (v if s["gs"] is None else v * s["gs"]).to(torch.bfloat16)


def _mm(s):
    c = s["case"]
    y = _values(s["a"], s["asf"], c["fmt"]) @ _values(s["b"], s["bsf"], c["fmt"]).t()
    return (y if s["ags"] is None else y * (s["ags"] * s["bgs"])).to(torch.bfloat16)


def _lowest_first(key, k):
    """Indices of the k largest of each row, equal ones by the lowest index."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]


def _route(s):
    c = s["case"]
    t, e, k, groups = c["t"], c["e"], c["k"], c["groups"]
    l = s["logits"].double()
    score = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
    key = l if s["bias"] is None else score + s["bias"].double()  # both scores grow with the logit
    if groups > 1:
        in_group = key.view(t, groups, -1)
        best = in_group.amax(2) if s["bias"] is None else in_group.topk(min(2, e // groups), 2).values.sum(2)
        keep = torch.zeros(t, groups, dtype=torch.bool, device=l.device).scatter_(1, _lowest_first(best, c["topg"]), True)
        key = key.masked_fill(~keep.repeat_interleave(e // groups, 1), -math.inf)
    ids = _lowest_first(key, k)
    w = score.gather(1, ids)
    return (w / w.sum(1, keepdim=True) if c["renorm"] else w).float(), ids.to(torch.int32)


def _experts(s):
    c = s["case"]
    t, k, h, fmt = c["t"], c["k"], c["h"], c["fmt"]
    flat = s["ids"].flatten().long()
    used, which = torch.unique(flat, return_inverse=True)  # the experts that have rows, and each row's among them
    order = torch.sort(which, stable=True).indices
    count = torch.bincount(which, minlength=used.numel())
    first = count.cumsum(0) - count
    at = torch.empty_like(flat)  # a row's place in its expert
    at[order] = torch.arange(flat.numel(), device=flat.device) - first[which[order]]
    room = int(count.max())

    def product(rows, w, sf, gw, ga):  # rows [T k, cols] quantised in turn, each times its expert's matrix
        code, asf = _quantise(rows, fmt, ga)
        v = _values(_pack(code), _store_scales(asf, fmt), fmt)
        padded = v.new_zeros(used.numel(), room, v.shape[1])
        padded[which, at] = v
        y = torch.bmm(padded, _values(w[used], sf[used], fmt).transpose(1, 2))
        y = y if gw is None else y * (gw[used] * ga).view(-1, 1, 1)
        return y[which, at]

    gate, up = product(s["x"].float().repeat_interleave(k, 0), s["w13"], s["w13_sf"], s["g13"], s["gx"]).chunk(2, 1)
    y = product(gate / (1 + torch.exp(-gate)) * up, s["w2"], s["w2_sf"], s["g2"], s["gh"])
    return (y.view(t, k, h) * s["weights"].unsqueeze(2)).sum(1).to(torch.bfloat16)


def run(state):
    if own:
        return _own(state)
    return {"quant": _quant, "mm": _mm, "route": _route, "experts": _experts}[state["case"]["op"]](state)


# -------------------------------------------------------------------------- the framework's operators
def _own(s):
    import fp8_quantized_linear_rms_b200 as fq
    c = s["case"]
    if c["op"] == "quant":
        if c["kind"] == "rmsnorm":
            q, sf = fq.fp8q_rmsnorm_fp4_quant(s["x"], s["w"], 1e-6, c["fmt"], gscale=s["gs"])
        elif c["kind"] == "silu":
            q, sf = fq.fp8q_silu_mul_fp4_quant(s["x"], c["fmt"], gscale=s["gs"])
        else:
            q, sf = fq.fp8q_fp4_quant(s["x"], c["fmt"], gscale=s["gs"])
        return fq.fp8q_fp4_dequant(q, sf, c["fmt"], gscale=s["gs"])
    if c["op"] == "mm":
        return fq.fp8q_scaled_mm_fp4(s["a"], s["b"], s["asf"], s["bsf"], c["fmt"], a_gscale=s["ags"], b_gscale=s["bgs"])
    if c["op"] == "route":
        return fq.fp8q_moe_route(s["logits"], c["k"], c["scoring"], bias=s["bias"], num_groups=c["groups"], topk_groups=c["topg"], renormalize=c["renorm"])
    return fq.fp8q_moe_experts_fp4(s["x"], s["ids"], s["weights"], s["w13"], s["w13_sf"], s["w2"], s["w2_sf"], c["fmt"],
                                   x_gscale=s["gx"], w13_gscale=s["g13"], h_gscale=s["gh"], w2_gscale=s["g2"])


# --------------------------------------------------------------------------------- what a pass needs
def work(case):
    gr = GROUP[case.get("fmt", "nvfp4")]
    op = case["op"]
    if op == "quant":  # the input in, codes and scales out, and the values that they stand for
        m, k = case["m"], case["k"]
        wide = 2 * k if case["kind"] == "silu" else k
        return {"bytes": m * (2 * wide + k / 2 + k / gr + 2 * k) + (2 * k if case["kind"] == "rmsnorm" else 0), "flops": 0}
    if op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k / 2 + k / gr) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "route":
        return {"bytes": case["t"] * (case["e"] * (2 if case["bf16"] else 4) + 8 * case["k"]) + (4 * case["e"] if case["bias"] else 0), "flops": 0}
    t, e, k, h, i = (case[n] for n in ("t", "e", "k", "h", "i"))
    used = min(e, t * k)
    return {"bytes": used * 3 * h * i * (1 / 2 + 1 / gr) + 4 * t * h + 8 * t * k, "flops": 6 * t * k * h * i}


# ----------------------------------------------------------------------- the definition, in 64 bits
def _exact_decode(q, stored, fmt):
    """code * sf in 64 bits, from the bits: sign, two of exponent, one of mantissa; the scale byte of each group by its address."""
    rows, half = q.shape
    code = torch.empty(rows, 2 * half, dtype=torch.long, device=q.device)
    code[:, ::2], code[:, 1::2] = (q % 16).long(), (q // 16).long()
    exp, man = (code // 2) % 4, code % 2
    v = torch.where(exp == 0, man * 0.5, (1 + 0.5 * man.double()) * 2.0 ** (exp - 1).double())
    v = torch.where(code >= 8, -v, v)
    r = torch.arange(rows, device=q.device).view(-1, 1)
    j = torch.arange(2 * half // GROUP[fmt], device=q.device).view(1, -1)
    b = stored.flatten()[((r // 128) * stored.shape[-2] + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4].long()
    if fmt == "nvfp4":
        ex, ma = b // 8 % 16, (b % 8).double()
        sf = torch.where(ex == 0, ma / 8 * 2.0 ** -6, (1 + ma / 8) * 2.0 ** (ex - 7).double())
    else:
        sf = 2.0 ** (b - 127).double()
    return (v.view(rows, -1, GROUP[fmt]) * sf.unsqueeze(2)).view(rows, -1)


def _exact_nearest(v, grid):
    """v rounded to the nearest of an increasing grid, ties to the even index, saturating."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    up = torch.searchsorted(grid, v.abs().contiguous()).clamp(1, len(grid) - 1)
    lo, hi = grid[up - 1], grid[up]
    mid = (lo + hi) / 2
    a = v.abs()
    out = torch.where((a > mid) | ((a == mid) & (up % 2 == 0)), hi, lo)
    return torch.copysign(out, v)


E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _exact_requantised(y, fmt, gs):
    """The values that y (64 bits) is held as."""
    y3 = y.view(y.shape[0], -1, GROUP[fmt])
    amax = y3.abs().amax(2, keepdim=True)
    if fmt == "nvfp4":
        fl = lambda v: v.float().double()  # noqa: E731  the definition's roundings to fp32
        d = fl(_exact_nearest(fl(fl(amax / 6) / gs), E4M3) * gs)
    else:
        d = 2.0 ** torch.ceil(torch.log2(amax.clamp(min=1e-10) / 6))
    return torch.where(d > 0, _exact_nearest(torch.where(d > 0, y3 / d, y3).float().double(), E2M1) * d, 0.0).view_as(y)


def _exact_silu(h):
    half = h.shape[1] // 2
    return h[:, :half] * torch.sigmoid(h[:, :half]) * h[:, half:]


def exact(case, seed):
    s = prepare(case, seed)
    num = lambda v: 1.0 if v is None else v.double()  # noqa: E731
    if case["op"] == "quant":
        y = s["x"].double()
        if case["kind"] == "rmsnorm":
            y = (y * torch.rsqrt((y * y).sum(1, keepdim=True) / case["k"] + 1e-6)).to(torch.bfloat16).double()
            y = (y * s["w"].double()).to(torch.bfloat16).double()
        elif case["kind"] == "silu":
            y = _exact_silu(y).to(torch.bfloat16).double()
        return _exact_requantised(y, case["fmt"], num(s["gs"]))
    if case["op"] == "mm":
        a, b = (_exact_decode(s[n], s[n + "sf"], case["fmt"]) for n in "ab")
        return torch.einsum("mk,nk->mn", a, b) * num(s["ags"]) * num(s["bgs"])
    if case["op"] == "route":
        l = s["logits"].double()
        z = torch.exp(l - l.amax(1, keepdim=True))
        score = z / z.sum(1, keepdim=True) if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-l))
        key = score.clone() if s["bias"] is None else score + s["bias"].double()
        size = case["e"] // case["groups"]
        if case["groups"] > 1:
            top = key.view(case["t"], -1, size).sort(2, descending=True).values[:, :, :1 if s["bias"] is None else 2].sum(2)
            rank = torch.argsort(top, dim=1, descending=True, stable=True).argsort(1)
            key[(rank >= case["topg"]).repeat_interleave(size, 1)] = -math.inf
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, : case["k"]]
        w = torch.take_along_dim(score, ids, 1)
        return (w / w.sum(1, keepdim=True) if case["renorm"] else w), ids.to(torch.int32)
    y = torch.zeros(case["t"], case["h"], dtype=torch.float64, device="cuda")
    for e in range(case["e"]):
        tok, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if tok.numel():
            pick = lambda v: 1.0 if v is None else v[e].double()  # noqa: E731
            x = _exact_requantised(s["x"][tok].double(), case["fmt"], num(s["gx"]))
            h = x @ _exact_decode(s["w13"][e], s["w13_sf"][e], case["fmt"]).t() * pick(s["g13"])
            h = _exact_requantised(_exact_silu(h), case["fmt"], num(s["gh"]))
            o = h @ _exact_decode(s["w2"][e], s["w2_sf"][e], case["fmt"]).t() * pick(s["g2"])
            y.index_add_(0, tok, o * s["weights"][tok, slot].double().unsqueeze(1))
    return y
