"""Measured cases of the mixture-of-experts operators: routing, RMS norm and
quantisation to microscaled formats, products grouped by expert, combination.

`run` computes an operator either in its plain form (elementary torch
operations in 32 bits) or, where `own` is set, by the library's call.
"""
import math

import torch

own = False

HIDDEN = 7168         # the K of the library's decode and MX workloads
BLOCK = {"mxfp8_b32": 32, "mxfp8": 128, "mxfp4": 32, "mxfp4_fp8a": 32}
MODES = ("bf16", "mxfp8_b32", "mxfp8", "mxfp4", "mxfp4_fp8a")


# ------------------------------------------------------------------- cases

def listed():
    return [
        # router of one decoded token: latency alone counts
        dict(name="route_1x128", op="route", tokens=1, experts=128, top_k=8, type="f32", padded=0.0),
        # router of a prefill with padding tokens (rows that are masked whole)
        dict(name="route_16383x256", op="route", tokens=16383, experts=256, top_k=8, type="bf16", padded=0.05),
        # norm before the experts, one token and an odd prefill
        dict(name="norm_1x7168", op="norm", tokens=1, width=HIDDEN, mode="mxfp8_b32", residual=True, normed=True),
        dict(name="norm_8191x7168", op="norm", tokens=8191, width=HIDDEN, mode="mxfp8_b32", residual=True, normed=False),
        # gated activation of a prefill's expert rows on the way to 8 bits
        dict(name="swiglu_32761x2048", op="quantize", rows=32761, width=2048, mode="mxfp8_b32", act="swiglu"),
        # 4-bit activations of a decode batch and their product with 4-bit weights
        dict(name="fp4_16x16384x7168", op="fp4_product", rows=16, n=16384, width=HIDDEN),
        # experts' products: one token (8 experts of 64 with one row each) ...
        dict(name="experts_1_fp4w", op="experts", tokens=1, top_k=8, experts=64, n=4096, width=HIDDEN,
             mode="mxfp4_fp8a", gather=True),
        # ... a decode batch (about 8 ragged rows an expert), second projection: rows as they lie
        dict(name="experts_61_mxfp8", op="experts", tokens=61, top_k=8, experts=64, n=HIDDEN, width=2048,
             mode="mxfp8_b32", gather=False),
        # ... a short prefill in bf16 with few experts
        dict(name="experts_777_bf16", op="experts", tokens=777, top_k=2, experts=16, n=2048, width=4096,
             mode="bf16", gather=True),
        # ... and a long prefill in 4 bits
        dict(name="experts_4096_mxfp4", op="experts", tokens=4096, top_k=8, experts=64, n=4096, width=HIDDEN,
             mode="mxfp4", gather=True),
        # weighted sum of a token's experts: one token, and a prefill with padding tokens
        dict(name="combine_1x7168", op="combine", tokens=1, top_k=8, width=HIDDEN, padded=0.0),
        dict(name="combine_8191x7168", op="combine", tokens=8191, top_k=8, width=HIDDEN, padded=0.05),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "norm", "quantize", "fp4_product", "experts", "experts", "experts", "combine"))
    if op == "route":
        e = rng.choice((8, 16, 40, 60, 64, 72, 96, 128, 160, 200, 256, 320, 384, 512))
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=e, top_k=rng.randint(1, 8),
                    type=rng.choice(("f32", "bf16")), padded=rng.choice((0.0, 0.05, 0.5)))
    if op == "norm":
        mode = rng.choice(("bf16", "mxfp8_b32", "mxfp8"))
        return dict(op=op, tokens=_log(rng, 1, 8192), width=128 * _log(rng, 2, 64), mode=mode,
                    residual=rng.random() < 0.75, normed=mode != "bf16" and rng.random() < 0.5)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 32768), width=128 * _log(rng, 2, 32), mode=rng.choice(("mxfp8_b32", "mxfp8")),
                    act=rng.choice(("none", "swiglu")))
    if op == "fp4_product":
        return dict(op=op, rows=_log(rng, 1, 4096), n=128 * _log(rng, 2, 128), width=256 * _log(rng, 2, 28))
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 8191), top_k=rng.randint(1, 8), width=8 * _log(rng, 64, 896),
                    padded=rng.choice((0.0, 0.05)))
    e = rng.choice((8, 16, 24, 32, 48, 64))
    return dict(op=op, tokens=_log(rng, 1, 4096), top_k=rng.randint(1, 8), experts=e, n=128 * _log(rng, 2, 32),
                width=256 * _log(rng, 1, 28), mode=rng.choice(MODES), gather=rng.random() < 0.5)


def _row_bytes(mode, k):
    codes = {"bf16": 2 * k, "mxfp4": k / 2}.get(mode, k)
    return codes + (k / BLOCK[mode] if mode != "bf16" else 0)


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * e * (4 if case["type"] == "f32" else 2) + 16 * t * k + 4 * (e + 1), "flops": 6 * t * e}
    if op == "norm":
        t, w = case["tokens"], case["width"]
        b = 2 * t * w * (3 if case["residual"] else 1) + 2 * w
        b += t * _row_bytes(case["mode"], w) + (2 * t * w if case["normed"] else 0)
        return {"bytes": b, "flops": 8 * t * w}
    if op == "quantize":
        t, w = case["rows"], case["width"]
        gated = case["act"] == "swiglu"
        return {"bytes": 2 * t * w * (2 if gated else 1) + t * _row_bytes(case["mode"], w), "flops": t * w * (10 if gated else 4)}
    if op == "fp4_product":
        m, n, w = case["rows"], case["n"], case["width"]
        return {"bytes": 2 * m * w + n * _row_bytes("mxfp4", w) + 2 * m * n, "flops": 2 * m * n * w}
    if op == "experts":
        t, e, n, w = case["tokens"], case["experts"], case["n"], case["width"]
        k, mode = min(case["top_k"], e), case["mode"]
        used = e * (1 - (1 - k / e) ** t)  # experts with a row, were all alike
        wmode = "mxfp4" if mode == "mxfp4_fp8a" else mode
        a = (t if case["gather"] else t * k) * _row_bytes(mode, w)
        return {"bytes": a + used * n * _row_bytes(wmode, w) + 2 * t * k * n, "flops": 2 * t * k * n * w}
    t, k, w = case["tokens"], case["top_k"], case["width"]
    return {"bytes": 2 * t * k * w + 4 * t * w + 8 * t * k, "flops": 2 * t * k * w}


# ------------------------------------------- microscaled values, plain form

def _pow2(c):
    """2^(c - 127) of E8M0 codes (int32), in 32 bits."""
    return torch.where(c > 0, c << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _e8m0(amax, fmt):
    """E8M0 codes (int32): 127 + ceil(log2(amax / largest value of the format)),
    127 for zero, 255 where amax is not finite."""
    top, shift = (0.75, 2) if fmt == "e2m1" else (0.875, 8)  # 6 = 0.75 * 2^3, 448 = 0.875 * 2^9
    m, e = torch.frexp(amax)
    c = (127 + e.to(torch.int32) - 1 - shift + (m > top)).clamp(0, 254)
    c = torch.where(amax == 0, 127, c)
    return torch.where(torch.isfinite(amax), c, 255).to(torch.int32)


def _round_e2m1(v):
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(v / step) * step


def _quantize(x, mode):
    """(values in units of their block's scale: e4m3, or 32 bits for e2m1; E8M0 codes) of 32-bit x [rows][width]."""
    fmt = "e2m1" if mode == "mxfp4" else "e4m3"
    b = x.view(x.shape[0], -1, BLOCK[mode])
    c = _e8m0(b.abs().amax(2), fmt)
    v = b * torch.where(c < 255, _pow2((254 - c).clamp(min=0)), 0.0)[:, :, None]
    v = torch.where((c < 255)[:, :, None], v, 0.0).view(x.shape)
    return (v.to(torch.float8_e4m3fn) if fmt == "e4m3" else _round_e2m1(v)), c


def _scales(c):
    return c.to(torch.uint8).view(torch.float8_e8m0fnu)


def _e2m1_codes(v):
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
    code = torch.bucketize(v.abs().contiguous(), mag) | torch.where(v < 0, 8, 0)
    code = code.to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _encode(x, mode):
    """Operand of a product: (codes, E8M0 codes as bytes or None)."""
    if mode == "bf16":
        return x.to(torch.bfloat16), None
    v, c = _quantize(x, mode)
    return (_e2m1_codes(v) if mode == "mxfp4" else v.view(torch.uint8)), c.to(torch.uint8)


def _decode(codes, scales, mode):
    """32-bit values [rows][width] of an operand."""
    if mode == "bf16":
        return codes.float()
    if mode == "mxfp4":
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                             device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=-1).flatten(-2)
    else:
        v = codes.view(torch.float8_e4m3fn).float()
    s = _pow2(scales.to(torch.int32))
    return (v.unflatten(-1, (s.shape[-1], -1)) * s[..., None]).flatten(-2)


def _weight_mode(mode):
    return "mxfp4" if mode == "mxfp4_fp8a" else mode


# ------------------------------------------------------------------- inputs

def _activations(g, rows, width):
    """Normal values with a few channels of larger spread, as hidden states have."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    spread = torch.rand(width, generator=g, device="cuda")
    return x * torch.where(spread > 0.99, 8.0, 0.5 + spread)


def _choices(g, tokens, experts, k):
    """Experts picked by each token [tokens][k], some experts more popular than others."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    logits += 0.5 * torch.randn(experts, generator=g, device="cuda")
    return logits.topk(k, dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "route":
        t, e = case["tokens"], case["experts"]
        l = 2 * torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        if case["padded"]:
            l[torch.rand(t, generator=g, device="cuda") < case["padded"]] = -math.inf
        s["top_k"] = min(case["top_k"], e)
        s["logits"] = l if case["type"] == "f32" else l.to(torch.bfloat16)
    elif op == "norm":
        t, w = case["tokens"], case["width"]
        s["x"] = _activations(g, t, w).to(torch.bfloat16)
        s["r"] = (4 * torch.randn(t, w, generator=g, device="cuda")).to(torch.bfloat16) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(w, generator=g, device="cuda")).to(torch.bfloat16)
    elif op == "quantize":
        gated = case["act"] == "swiglu"
        s["x"] = _activations(g, case["rows"], case["width"] * (2 if gated else 1)).to(torch.bfloat16)
    elif op == "fp4_product":
        s["x"] = _activations(g, case["rows"], case["width"]).to(torch.bfloat16)
        s["w"], s["ws"] = _encode(torch.randn(case["n"], case["width"], generator=g, device="cuda"), "mxfp4")
        if own:
            import mx_gemm_gb300 as fg
            s["pb"] = fg.preshuffle_b("mxfp4", s["w"], s["ws"])
    elif op == "experts":
        t, e, n, w, mode = case["tokens"], case["experts"], case["n"], case["width"], case["mode"]
        k = min(case["top_k"], e)
        flat = _choices(g, t, e, k).flatten()
        order = torch.sort(flat, stable=True)
        s["offsets"] = torch.searchsorted(order.values, torch.arange(e + 1, device="cuda")).int()
        s["rows"] = (order.indices // k).int() if case["gather"] else None
        s["a"], s["as"] = _encode(_activations(g, t if case["gather"] else t * k, w), "mxfp8_b32" if mode == "mxfp4_fp8a" else mode)
        parts = [_encode(torch.randn(n, w, generator=g, device="cuda") / math.sqrt(w), _weight_mode(mode)) for _ in range(e)]
        s["w"] = torch.cat([p[0] for p in parts])
        s["ws"] = None if mode == "bf16" else torch.cat([p[1] for p in parts])
        s["total"] = t * k
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # rows of the busiest expert
        if own:
            import mx_gemm_gb300 as fg
            s["pb"] = fg.preshuffle_b(mode, s["w"], s["ws"])
    else:
        t, k, w = case["tokens"], case["top_k"], case["width"]
        s["y"] = torch.randn(t * k, w, generator=g, device="cuda").to(torch.bfloat16)
        s["r"] = (4 * torch.randn(t, w, generator=g, device="cuda")).to(torch.bfloat16)
        s["weights"] = torch.softmax(torch.randn(t, k, generator=g, device="cuda"), dim=1)
        slots = torch.randperm(t * k, generator=g, device="cuda").view(t, k).int()
        if case["padded"]:
            slots[torch.rand(t, generator=g, device="cuda") < case["padded"]] = -1
        s["slots"] = slots
    return s


# -------------------------------------------------------------- one pass

def _run_own(s):
    import mx_gemm_gb300 as fg
    op = s["op"]
    if op == "route":
        return tuple(fg.moe_route(s["logits"], s["top_k"]))
    if op == "norm":
        return tuple(fg.rmsnorm_quantize(s["mode"], s["x"], s["weight"], residual=s["r"], normed=s["normed"]))
    if op == "quantize":
        return fg.quantize(s["mode"], s["x"], act=s["act"])
    if op == "fp4_product":
        codes, scales = fg.quantize("mxfp4", s["x"])
        return fg.gemm(codes, s["pb"], scales)
    if op == "experts":
        return fg.grouped_gemm(s["a"], s["pb"], s["offsets"], s["as"], rows=s["rows"])
    return fg.moe_combine(s["y"], s["slots"], s["weights"], residual=s["r"])


def _route(s):
    l, k = s["logits"].float(), s["top_k"]
    t, e = l.shape
    l = torch.where(torch.isnan(l), -math.inf, l)
    top = torch.sort(l, dim=1, descending=True, stable=True)
    v, idx = top.values[:, :k], top.indices[:, :k]
    ok = v > -math.inf
    p = torch.where(ok, torch.exp(torch.where(v == v[:, :1], 0.0, v - v[:, :1])), 0.0)
    weights = torch.where(ok, p / p.sum(1, keepdim=True), 0.0)
    flat = torch.sort(torch.where(ok, idx, e).flatten(), stable=True)
    offsets = torch.searchsorted(flat.values, torch.arange(e + 1, device=l.device)).int()
    rows = torch.where(flat.values < e, flat.indices // k, -1).int()
    slots = torch.empty_like(flat.indices)
    slots[flat.indices] = torch.arange(t * k, device=l.device)
    slots = torch.where(ok, slots.view(t, k), -1).int()
    return weights, torch.where(ok, idx, -1).int(), offsets, rows, slots


def _norm(s):
    x = s["x"].float()
    h = x + s["r"].float() if s["residual"] else x
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    codes = scales = None
    if s["mode"] != "bf16":
        codes, c = _quantize(y, s["mode"])
        scales = _scales(c)
    return (codes, scales, h.to(torch.bfloat16) if s["residual"] else None,
            y.to(torch.bfloat16) if s["normed"] or s["mode"] == "bf16" else None)


def _run_plain(s):
    op = s["op"]
    if op == "route":
        return _route(s)
    if op == "norm":
        return _norm(s)
    if op == "quantize":
        x = s["x"].float()
        if s["act"] == "swiglu":
            gate, up = x.chunk(2, dim=1)
            x = gate / (1 + torch.exp(-gate)) * up
        v, c = _quantize(x, s["mode"])
        return v, _scales(c)
    if op == "fp4_product":
        v, c = _quantize(s["x"].float(), "mxfp4")
        a = (v.unflatten(1, (c.shape[1], -1)) * _pow2(c)[:, :, None]).flatten(1)
        return (a @ _decode(s["w"], s["ws"], "mxfp4").T).to(torch.bfloat16)
    if op == "experts":
        e, n, total, most, mode = s["experts"], s["n"], s["total"], s["most"], s["mode"]
        a = _decode(s["a"], s["as"], "mxfp8_b32" if mode == "mxfp4_fp8a" else mode)
        at = torch.arange(total, device=a.device)
        expert = torch.searchsorted(s["offsets"], at, right=True, out_int32=True) - 1
        a = a[s["rows"]] if s["gather"] else a
        w = s["w"].view(e, n, -1)
        ws = None if s["ws"] is None else s["ws"].view(e, n, -1)
        if total <= e:  # few rows: each with its own expert's weight
            w = _decode(w[expert], None if ws is None else ws[expert], _weight_mode(mode))
            return (w @ a[:, :, None])[:, :, 0].to(torch.bfloat16)
        place = at - s["offsets"][expert]
        padded = torch.zeros(e, most, a.shape[1], device=a.device)
        padded[expert, place] = a
        y = padded @ _decode(w, ws, _weight_mode(mode)).transpose(1, 2)
        return y[expert, place].to(torch.bfloat16)
    ok = s["slots"] >= 0
    y = s["y"][s["slots"].clamp(min=0)].float() * torch.where(ok, s["weights"], 0.0)[:, :, None]
    return (s["r"].float() + y.sum(1)).to(torch.bfloat16)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------- the definitions in 64 bits

def _table(exp_bits, man_bits, bias):
    """Values of a small floating format's codes, without its not-a-numbers."""
    vals = []
    for code in range(1 << (1 + exp_bits + man_bits)):
        e = (code >> man_bits) & ((1 << exp_bits) - 1)
        m = (code & ((1 << man_bits) - 1)) / (1 << man_bits)
        v = (1 + m) * 2.0 ** (e - bias) if e else m * 2.0 ** (1 - bias)
        vals.append(-v if code >> (exp_bits + man_bits) else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _values64(codes, scales, mode):
    if mode == "bf16":
        return codes.double()
    if mode == "mxfp4":
        c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.int64, device=codes.device)
        c[:, 0::2] = codes % 16
        c[:, 1::2] = codes // 16
        v = _table(2, 1, 1)[c]
    else:
        v = _table(4, 3, 7)[codes.long()]
    per = v.shape[1] // scales.shape[1]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(per, dim=1)


def _in_blocks64(v, mode):
    """v over its blocks' scales, not rounded, and the scales as exponents of two."""
    top = 6.0 if mode == "mxfp4" else 448.0
    b = v.unflatten(1, (-1, BLOCK[mode]))
    amax = b.abs().amax(2)
    # the smallest whole e with amax <= top * 2^e, mended where the logarithm's rounding is off by one
    e = torch.where(amax > 0, torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / top)), 0.0)
    e = torch.where(amax > top * torch.exp2(e), e + 1, e)
    e = torch.where((amax > 0) & (amax <= top * torch.exp2(e - 1)), e - 1, e).clamp(-127, 127)
    return (b / torch.exp2(e)[:, :, None]).flatten(1), e


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        l = s["logits"].double()
        top = torch.topk(l, s["top_k"], dim=1).values
        w = torch.softmax(top, dim=1)
        return torch.where(torch.isfinite(top), w, 0.0), None, None, None, None
    if op == "norm":
        h = s["x"].double() + (s["r"].double() if case["residual"] else 0)
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / h.shape[1] + 1e-6) * s["weight"].double()
        mx = case["mode"] != "bf16"
        return (_in_blocks64(y, case["mode"])[0] if mx else None, None, h if case["residual"] else None,
                y if case["normed"] or not mx else None)
    if op == "quantize":
        v = s["x"].double()
        if case["act"] == "swiglu":
            w = case["width"]
            v = v[:, :w] * torch.sigmoid(v[:, :w]) * v[:, w:]
        return _in_blocks64(v, case["mode"])[0], None
    if op == "fp4_product":
        v, e = _in_blocks64(s["x"].double(), "mxfp4")
        grid = _table(2, 1, 1)[:8]
        mid = (grid[1:] + grid[:-1]) / 2
        a = v.abs().contiguous()
        lo, hi = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # they differ at a tie: the even code
        q = torch.sign(v) * grid[torch.where(lo % 2 == 0, lo, hi)]
        q = q * torch.exp2(e).repeat_interleave(32, dim=1)
        return q @ _values64(s["w"], s["ws"], "mxfp4").T
    if op == "experts":
        mode, n, cuts = case["mode"], case["n"], s["offsets"].tolist()
        a = _values64(s["a"], s["as"], "mxfp8_b32" if mode == "mxfp4_fp8a" else mode)
        out = torch.empty(s["total"], n, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            i, j = cuts[e], cuts[e + 1]
            if i < j:
                mine = a[s["rows"][i:j].long()] if case["gather"] else a[i:j]
                ws = None if s["ws"] is None else s["ws"][e * n:(e + 1) * n]
                out[i:j] = mine @ _values64(s["w"][e * n:(e + 1) * n], ws, _weight_mode(mode)).T
        return out
    out = s["r"].double()
    for j in range(case["top_k"]):
        slot = s["slots"][:, j].long()
        out += torch.where(slot >= 0, s["weights"][:, j].double(), 0.0)[:, None] * s["y"][slot.clamp(min=0)].double()
    return out
