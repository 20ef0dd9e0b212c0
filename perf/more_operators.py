"""Measured cases of training a mixture-of-experts layer in 8 bits: the weights'
quantisation in 128 x 128 blocks and the experts' products with them, the gated
activation with an 8-bit checkpoint and its backward pass, the weights' gradients,
and the router's balance loss and gradient.

`run` computes an operator either in its plain form (elementary torch
operations in 32 bits) or, where `own` is set, by the library's calls.
"""
import math

import torch

own = False

MODES = ("mxfp8_b32", "mxfp8", "fp8_block128")
BLOCK = {"mxfp8_b32": 32, "mxfp8": 128, "fp8_block128": 128}
TILE = 128   # rows of an expert that a slab of a column operand holds


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one small weight after an optimiser's step; and eight experts' up-projections, transposed for the input's gradient
        dict(name="weight_1x256x512", op="weight", experts=1, n=256, k=512, type="f32", transpose=False),
        dict(name="weight_8x4096x7168_t", op="weight", experts=8, n=4096, k=7168, type="bf16", transpose=True),
        # experts' products with fp32 block scales: a short batch, ragged, and a long one gathered by token
        dict(name="experts_777", op="experts", tokens=777, top_k=2, experts=16, n=2048, k=4096, gather=False),
        dict(name="experts_4096", op="experts", tokens=4096, top_k=8, experts=64, n=4096, k=7168, gather=True),
        # gated activation with its checkpoint: one token's experts, and a long batch
        dict(name="checkpoint_8x2048", op="checkpoint", rows=8, width=2048, mode="mxfp8_b32"),
        dict(name="checkpoint_32761x2048", op="checkpoint", rows=32761, width=2048, mode="mxfp8_b32"),
        # its backward pass from the checkpoint: few experts with ragged rows, and a long batch with padding tokens
        dict(name="swiglu_grad_777x2", op="swiglu_grad", tokens=777, top_k=2, experts=16, width=1024, mode="fp8_block128", padded=0.0),
        dict(name="swiglu_grad_4095x8", op="swiglu_grad", tokens=4095, top_k=8, experts=64, width=2048, mode="mxfp8_b32", padded=0.05),
        # weights' gradient from the layer's 8-bit input and the output's gradient: small experts, and large ones
        dict(name="weight_grad_777x2", op="weight_grad", tokens=777, top_k=2, experts=16, n=512, k=1024, mode="fp8_block128", out="f32"),
        dict(name="weight_grad_4096x8", op="weight_grad", tokens=4096, top_k=8, experts=16, n=4096, k=7168, mode="mxfp8_b32", out="f32"),
        # router: balance loss, counts and the logits' gradient of a small batch and of a long one with padding tokens
        dict(name="router_61x64", op="router", tokens=61, experts=64, top_k=8, type="f32", padded=0.0, renormalize=True),
        dict(name="router_16383x256", op="router", tokens=16383, experts=256, top_k=8, type="bf16", padded=0.05, renormalize=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("weight", "experts", "experts", "checkpoint", "swiglu_grad", "swiglu_grad", "weight_grad", "weight_grad", "router"))
    if op == "weight":
        return dict(op=op, experts=rng.randint(1, 8), n=128 * _log(rng, 1, 32), k=128 * _log(rng, 1, 56),
                    type=rng.choice(("f32", "bf16")), transpose=rng.random() < 0.5)
    if op == "experts":
        return dict(op=op, tokens=_log(rng, 16, 4096), top_k=rng.randint(1, 8), experts=rng.choice((8, 16, 24, 32, 48, 64)),
                    n=128 * _log(rng, 2, 32), k=128 * _log(rng, 1, 56), gather=rng.random() < 0.5)
    if op == "checkpoint":
        return dict(op=op, rows=_log(rng, 1, 32768), width=128 * _log(rng, 1, 16), mode=rng.choice(MODES))
    if op == "swiglu_grad":
        return dict(op=op, tokens=_log(rng, 1, 4096), top_k=rng.randint(1, 8), experts=rng.choice((8, 16, 24, 40, 64)),
                    width=128 * _log(rng, 1, 16), mode=rng.choice(MODES), padded=rng.choice((0.0, 0.05)))
    if op == "weight_grad":
        return dict(op=op, tokens=_log(rng, 1, 4096), top_k=rng.randint(1, 8), experts=rng.choice((8, 12, 16)),
                    n=128 * _log(rng, 1, 32), k=128 * _log(rng, 1, 56), mode=rng.choice(MODES + ("bf16",)),
                    out=rng.choice(("f32", "bf16")))
    return dict(op=op, tokens=_log(rng, 1, 16384), experts=rng.choice((8, 16, 40, 60, 64, 72, 96, 128, 160, 256, 384, 512)),
                top_k=rng.randint(1, 8), type=rng.choice(("f32", "bf16")), padded=rng.choice((0.0, 0.05, 0.5)),
                renormalize=rng.random() < 0.7)


def _codes_bytes(mode, count):
    """Bytes of `count` values in a format: codes and scales."""
    return 2 * count if mode == "bf16" else count * (1 + (4 if mode == "fp8_block128" else 1) / BLOCK[mode])


def _capacity(rows, experts):
    """Rows that a column operand holds for `rows` rows, however they fall on the experts."""
    return TILE * max(1, rows // TILE + min(experts, rows))


def work(case):
    op = case["op"]
    if op == "weight":
        count = case["experts"] * case["n"] * case["k"]
        return {"bytes": count * (4 if case["type"] == "f32" else 2) + count + count / 4096, "flops": 2 * count}
    if op == "checkpoint":
        count = case["rows"] * case["width"]
        return {"bytes": 4 * count + 3 * _codes_bytes(case["mode"], count), "flops": 14 * count}
    t, e = case["tokens"], case["experts"]
    k = min(case["top_k"], e)
    if op == "router":
        return {"bytes": 2 * t * e * (4 if case["type"] == "f32" else 2) + 12 * t * k + 16 * e, "flops": 12 * t * e}
    used = e * (1 - (1 - k / e) ** t)  # experts with a row, were all alike
    if op == "experts":
        n, w = case["n"], case["k"]
        a = (t if case["gather"] else t * k) * w * (1 + 4 / 128)
        return {"bytes": a + used * n * w + 2 * t * k * n, "flops": 2 * t * k * n * w}
    if op == "swiglu_grad":
        count = t * k * case["width"]
        return {"bytes": 2 * count + 4 * _codes_bytes(case["mode"], count) + 3 * count * (1 + 1 / 32) + 12 * t * k, "flops": 30 * count}
    n, w = case["n"], case["k"]
    return {"bytes": _codes_bytes(case["mode"], t * w) + 2 * t * k * n + (4 if case["out"] == "f32" else 2) * e * n * w,
            "flops": 2 * t * k * n * w}


# ---------------------------------------------------- 8-bit values, plain form

def _pow2(c):
    """2^(c - 127) of E8M0 codes (int32), in 32 bits."""
    return torch.where(c > 0, c << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _e8m0(amax):
    """E8M0 codes (int32): 127 + ceil(log2(amax / 448)), 127 for zero, 255 where amax is not finite."""
    m, e = torch.frexp(amax)  # 448 = 0.875 * 2^9
    c = (127 + e.to(torch.int32) - 9 + (m > 0.875)).clamp(0, 254)
    c = torch.where(amax == 0, 127, c)
    return torch.where(torch.isfinite(amax), c, 255).to(torch.int32)


def _quantize(x, mode):
    """(e4m3 codes, scales) of 32-bit x [rows][width] in blocks along the rows."""
    b = x.unflatten(1, (-1, BLOCK[mode]))
    amax = b.abs().amax(2)
    if mode == "fp8_block128":
        s = torch.where(amax == 0, 1.0, amax / 448)
        return (b / s[:, :, None]).flatten(1).to(torch.float8_e4m3fn), s
    c = _e8m0(amax)
    v = (b * _pow2((254 - c).clamp(min=0))[:, :, None]).flatten(1)
    return v.to(torch.float8_e4m3fn), c.to(torch.uint8).view(torch.float8_e8m0fnu)


def _decode(codes, scales):
    """32-bit values [rows][width] of codes and scales (E8M0 or fp32)."""
    s = scales if scales.dtype == torch.float32 else _pow2(scales.view(torch.uint8).to(torch.int32))
    return (codes.float().unflatten(1, (s.shape[1], -1)) * s[:, :, None]).flatten(1)


def _places(offsets, rows, experts):
    """Row of each place of a column operand, and whether there is one."""
    tiles = (offsets[1:] - offsets[:-1] + TILE - 1) // TILE
    ends = torch.cumsum(tiles, 0)
    at = torch.arange(_capacity(rows, experts), device=offsets.device)
    e = torch.searchsorted(ends, at // TILE, right=True).clamp(max=experts - 1)
    row = offsets[e] + (at // TILE - (ends - tiles)[e]) * TILE + at % TILE
    return row.clamp(max=rows - 1), (row < offsets[e + 1]) & (at // TILE < ends[-1])


def _columns(x, place, there):
    """(codes, E8M0 codes as int32) [C][P] of 32-bit x [rows][C], transposed, in blocks of 32 places."""
    v = torch.where(there[:, None], x[place], 0.0).T.unflatten(1, (-1, 32))
    c = _e8m0(v.abs().amax(2))
    return (v * _pow2(254 - c)[:, :, None]).flatten(1).to(torch.float8_e4m3fn), c


def _image(codes):
    """The slabs of [C][P] codes: 128 x 128 each, 16-byte piece i of row r at i ^ (r % 8)."""
    c, p = codes.shape
    b = codes.view(torch.uint8).view(c // 128, 128, p // 128, 8, 16).transpose(1, 2)
    r = torch.arange(128, device=codes.device)[:, None]
    to = torch.arange(8, device=codes.device)[None, :] ^ (r % 8)
    return b[:, :, r, to].flatten().view(torch.float8_e4m3fn)


def _atoms(c):
    """The scale atoms of [C][P / 32] E8M0 codes: byte 16 (r % 32) + 4 (r / 32) + j of a slab's 512."""
    n, p = c.shape
    b = c.to(torch.uint8).view(n // 128, 4, 32, p // 4, 4).permute(0, 3, 2, 1, 4)
    return b.flatten().view(torch.float8_e8m0fnu)


# ------------------------------------------------------------------- inputs

def _activations(g, rows, width):
    """Normal values with a few channels of larger spread, as hidden states have."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    spread = torch.rand(width, generator=g, device="cuda")
    return x * torch.where(spread > 0.99, 8.0, 0.5 + spread)


def _routing(g, tokens, experts, k, padded, logits=None, renormalize=True):
    """What routing gives: weights, experts, offsets, rows, slots; `padded`: share of tokens with no choice."""
    if logits is None:
        logits = torch.randn(tokens, experts, generator=g, device="cuda") + 0.5 * torch.randn(experts, generator=g, device="cuda")
        if padded:
            logits[torch.rand(tokens, generator=g, device="cuda") < padded] = -math.inf
    l = logits.float()
    top = torch.sort(l, dim=1, descending=True, stable=True)
    v, idx = top.values[:, :k], top.indices[:, :k]
    ok = v > -math.inf
    p = torch.where(ok, torch.exp(torch.where(ok, v - l.amax(1, keepdim=True), 0.0)), 0.0)
    total = p.sum(1, keepdim=True) if renormalize else torch.where(l > -math.inf, torch.exp(l - l.amax(1, keepdim=True)), 0.0).sum(1, keepdim=True)
    weights = torch.where(ok, p / total, 0.0)
    flat = torch.sort(torch.where(ok, idx, experts).flatten(), stable=True)
    offsets = torch.searchsorted(flat.values, torch.arange(experts + 1, device="cuda")).int()
    rows = torch.where(flat.values < experts, flat.indices // k, -1).int()
    slots = torch.empty_like(flat.indices)
    slots[flat.indices] = torch.arange(tokens * k, device="cuda")
    slots = torch.where(ok, slots.view(tokens, k), -1).int()
    return weights, torch.where(ok, idx, -1).int(), offsets, rows, slots


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "weight":
        w = torch.randn(case["experts"], case["n"], case["k"], generator=g, device="cuda") / math.sqrt(case["k"])
        s["w"] = w if case["type"] == "f32" else w.to(torch.bfloat16)
        return s
    if op == "checkpoint":
        s["x"] = _activations(g, case["rows"], 2 * case["width"]).to(torch.bfloat16)
        return s
    t, e = case["tokens"], case["experts"]
    s["top_k"] = k = min(case["top_k"], e)
    if op == "router":
        l = 2 * torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        if case["padded"]:
            l[torch.rand(t, generator=g, device="cuda") < case["padded"]] = -math.inf
            l[0, 0] = 0.0  # (a batch has a token)
        s["logits"] = l if case["type"] == "f32" else l.to(torch.bfloat16)
        s["routing"] = _routing(g, t, e, k, 0.0, s["logits"], case["renormalize"])
        s["dweights"] = torch.randn(t, k, generator=g, device="cuda")
        s["coefficient"] = 0.01
        return s
    s["routing"] = _routing(g, t, e, k, case.get("padded", 0.0))
    if op == "experts":
        n, w = case["n"], case["k"]
        s["a"], s["as"] = _quantize(_activations(g, t if case["gather"] else t * k, w), "fp8_block128")
        s["w"] = torch.empty(e * n, w, dtype=torch.float8_e4m3fn, device="cuda")
        s["ws"] = torch.empty(e * n // 128, w // 128, device="cuda")
        for i in range(e):
            b = torch.randn(n, w, generator=g, device="cuda").div_(math.sqrt(w)).view(n // 128, 128, w // 128, 128)
            top = b.abs().amax((1, 3)) / 448
            s["w"][i * n:(i + 1) * n] = (b / top[:, None, :, None]).view(n, w).to(torch.float8_e4m3fn)
            s["ws"][i * n // 128:(i + 1) * n // 128] = top
        offsets = s["routing"][2]
        s["most"] = int((offsets[1:] - offsets[:-1]).max())  # rows of the busiest expert
        if own:
            import mx_gemm_gb300 as fg
            s["pb"] = fg.preshuffle_b("fp8_block128", s["w"], s["ws"])
    elif op == "swiglu_grad":
        up = _activations(g, t * k, 2 * case["width"]).to(torch.bfloat16)
        s["saved"], s["saved_scales"] = _quantize(up.float(), case["mode"])
        s["dy"] = (0.01 * torch.randn(t * k, case["width"], generator=g, device="cuda")).to(torch.bfloat16)
    else:
        x = _activations(g, t, case["k"]).to(torch.bfloat16)
        s["x"], s["xs"] = (x, None) if case["mode"] == "bf16" else _quantize(x.float(), case["mode"])
        s["dy"] = (0.01 * torch.randn(t * k, case["n"], generator=g, device="cuda")).to(torch.bfloat16)
        offsets = s["routing"][2]
        s["most"] = int((offsets[1:] - offsets[:-1]).max())
    return s


# -------------------------------------------------------------- one pass

def _run_own(s):
    import mx_gemm_gb300 as fg
    op = s["op"]
    if op == "weight":
        return fg.quantize_weight("fp8_block128", s["w"], transpose=s["transpose"])
    if op == "checkpoint":
        return fg.swiglu_checkpoint(s["mode"], s["x"])
    r = fg.Routing(*s["routing"])
    if op == "router":
        b = fg.moe_balance_loss(s["logits"], r.offsets, s["coefficient"])
        d = fg.moe_route_backward(s["logits"], r, s["dweights"], slopes=b.slopes, renormalize=s["renormalize"])
        return b.loss, b.counts, b.probs, d
    if op == "experts":
        return fg.grouped_gemm(s["a"], s["pb"], r.offsets, s["as"], rows=r.rows if s["gather"] else None)
    if op == "swiglu_grad":
        d = fg.swiglu_backward(s["mode"], s["dy"], s["saved"], s["saved_scales"], routing=r, columns=True)
        return (d.codes, d.scales, d.dweights, d.dx_columns.data.view(torch.float8_e4m3fn), d.dx_columns.sf.view(torch.float8_e8m0fnu),
                d.act_columns.data.view(torch.float8_e4m3fn), d.act_columns.sf.view(torch.float8_e8m0fnu))
    x = fg.quantize_columns(s["x"], r.offsets, scales=s["xs"], rows=r.rows)
    dy = fg.quantize_columns(s["dy"], r.offsets)
    return fg.grouped_wgrad(dy, x, r.offsets, dtype=torch.float32 if s["out"] == "f32" else torch.bfloat16)


def _softmax(l):
    """(p, tokens that have a logit to pick) of 32-bit logits; rows of -infinity have p = 0."""
    top = l.amax(1, keepdim=True)
    some = top > -math.inf
    p = torch.where(l > -math.inf, torch.exp(l - torch.where(some, top, 0.0)), 0.0)
    return torch.where(some, p / p.sum(1, keepdim=True), 0.0), some.sum()


def _router(s):
    l, e = s["logits"].float(), s["experts"]
    weights, chosen, offsets, _, _ = s["routing"]
    p, tokens = _softmax(l)
    counts = offsets[1:] - offsets[:-1]
    f = counts.float() / offsets[-1]
    probs = p.sum(0) / tokens
    loss = s["coefficient"] * e * (f * probs).sum()
    slopes = s["coefficient"] * e * f / tokens
    d = p * (slopes - (p * slopes).sum(1, keepdim=True))
    ok = chosen >= 0
    dw = torch.where(ok, s["dweights"], 0.0)
    at = chosen.clamp(min=0).long()
    if s["renormalize"]:
        q = torch.where(ok, torch.gather(p, 1, at), 0.0)
        total = q.sum(1, keepdim=True)
        q = torch.where(total > 0, q / total, 0.0)
        d = d.scatter_add(1, at, q * (dw - (q * dw).sum(1, keepdim=True)))
    else:
        q = torch.where(ok, torch.gather(p, 1, at), 0.0)
        d = d.scatter_add(1, at, q * dw) - p * (q * dw).sum(1, keepdim=True)
    return loss, counts, probs, d.to(s["logits"].dtype)


def _padded(x, offsets, experts, most):
    """Rows of each expert next to one another, [E][most][...], zeros behind them."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device)
    ok = at < offsets[1:, None]
    return torch.where(ok[:, :, None], x[at.clamp(max=x.shape[0] - 1)], 0.0)


def _run_plain(s):
    op = s["op"]
    if op == "weight":
        w = s["w"].float()
        w = w.transpose(1, 2) if s["transpose"] else w
        n, k = w.shape[1:]
        b = w.reshape(-1, 128, k // 128, 128)
        top = b.abs().amax((1, 3))
        top = torch.where(top == 0, 1.0, top / 448)
        return (b / top[:, None, :, None]).view(-1, k).to(torch.float8_e4m3fn), top
    if op == "checkpoint":
        x = s["x"].float()
        gate, up = x.chunk(2, dim=1)
        return _quantize(gate / (1 + torch.exp(-gate)) * up, s["mode"]) + _quantize(x, s["mode"])
    if op == "router":
        return _router(s)
    weights, _, offsets, rows, slots = s["routing"]
    e, t, k = s["experts"], s["tokens"], s["top_k"]
    total = t * k
    if op == "experts":
        n, at = s["n"], torch.arange(total, device=offsets.device)
        a = _decode(s["a"], s["as"])
        a = a[rows] if s["gather"] else a
        w = (s["w"].float().view(-1, 128, s["k"] // 128, 128) * s["ws"][:, None, :, None]).view(e, n, -1)
        y = _padded(a, offsets, e, s["most"]) @ w.transpose(1, 2)
        expert = torch.searchsorted(offsets, at, right=True, out_int32=True) - 1
        return y[expert, at - offsets[expert]].to(torch.bfloat16)
    place, there = _places(offsets, total, e)
    if op == "swiglu_grad":
        gate, up = _decode(s["saved"], s["saved_scales"]).chunk(2, dim=1)
        dy = s["dy"].float()
        routed = (torch.arange(total, device=dy.device) < offsets[-1])[:, None]
        by_slot = torch.zeros(total + 1, device=dy.device)
        by_slot[torch.where(slots >= 0, slots, total).long()] = weights
        sig = 1 / (1 + torch.exp(-gate))
        act = gate * sig * up
        dots = torch.where(routed, dy * act, 0.0).sum(1)
        dweights = torch.where(slots >= 0, dots[slots.clamp(min=0)], 0.0)
        w = by_slot[:total, None]
        dy = dy * w
        dx = torch.cat([dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig], dim=1)
        codes, scales = _quantize(torch.where(routed, dx, 0.0), s["mode"])
        dx_codes, dx_scales = _columns(dx, place, there)
        act_codes, act_scales = _columns(w * act, place, there)
        return codes, scales, dweights, _image(dx_codes), _atoms(dx_scales), _image(act_codes), _atoms(act_scales)
    x = s["x"].float() if s["xs"] is None else _decode(s["x"], s["xs"])
    x, xc = _columns(x[rows], place, there)
    dy, dyc = _columns(s["dy"].float(), place, there)
    # the columns' values by place again: [P][C]
    x = (x.float().unflatten(1, (-1, 32)) * _pow2(xc)[:, :, None]).flatten(1).T
    dy = (dy.float().unflatten(1, (-1, 32)) * _pow2(dyc)[:, :, None]).flatten(1).T
    tiles = (offsets[1:] - offsets[:-1] + TILE - 1) // TILE
    starts = TILE * torch.cat([tiles.new_zeros(1), torch.cumsum(tiles, 0)])
    dw = _padded(dy, starts, e, -(-s["most"] // TILE) * TILE).transpose(1, 2) @ _padded(x, starts, e, -(-s["most"] // TILE) * TILE)
    return dw if s["out"] == "f32" else dw.to(torch.bfloat16)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------- the definitions in 64 bits

def _block_exponent64(b):
    """Smallest whole e with max |b| <= 448 * 2^e over the last axis (0 for zeros)."""
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 448)), 0.0)
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)  # the logarithm's rounding, mended
    return torch.where((amax > 0) & (amax <= 448 * torch.exp2(e - 1)), e - 1, e).clamp(-127, 127)


def _over_scales64(v, mode):
    """v over its blocks' scales, not rounded; and the scales."""
    b = v.unflatten(1, (-1, BLOCK[mode]))
    if mode == "fp8_block128":
        s = b.abs().amax(2) / 448
        s = torch.where(s > 0, s, 1.0)
    else:
        s = torch.exp2(_block_exponent64(b))
    return (b / s[:, :, None]).flatten(1), s


def _values64(codes, scales):
    s = scales.double() if scales.dtype == torch.float32 else torch.exp2(scales.view(torch.uint8).double() - 127)
    return codes.double() * s.repeat_interleave(codes.shape[1] // s.shape[1], dim=1)


def _e4m3_64(v):
    """Nearest e4m3 value, ties to even, |v| <= 448."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6) - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _as_images64(parts, capacity):
    """Slabs and atoms of an operand from each expert's rows [count][C], not rounded, over their blocks' scales."""
    c = parts[0].shape[1]
    v = torch.zeros(c, capacity, dtype=torch.float64, device=parts[0].device)
    at = 0
    for x in parts:
        v[:, at:at + x.shape[0]] = x.T
        at += -(-x.shape[0] // TILE) * TILE
    b = v.unflatten(1, (-1, 32))
    s = torch.exp2(_block_exponent64(b))
    q = (b / s[:, :, None]).reshape(c // 128, 128, capacity // 128, 128).transpose(1, 2).clone()
    for r in range(8):
        mine = q[:, :, r::8].unflatten(3, (8, 16))
        q[:, :, r::8] = mine[:, :, :, [i ^ r for i in range(8)]].flatten(3)
    return q.flatten()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "weight":
        w = s["w"].double().transpose(1, 2) if case["transpose"] else s["w"].double()
        k = w.shape[2]
        b = w.reshape(-1, 128, k // 128, 128)
        top = b.abs().amax((1, 3)) / 448
        top = torch.where(top > 0, top, 1.0)
        return (b / top[:, None, :, None]).reshape(-1, k), top
    if op == "checkpoint":
        x, w = s["x"].double(), case["width"]
        fp32 = case["mode"] == "fp8_block128"
        a, b = _over_scales64(x[:, :w] * torch.sigmoid(x[:, :w]) * x[:, w:], case["mode"]), _over_scales64(x, case["mode"])
        return a[0], a[1] if fp32 else None, b[0], b[1] if fp32 else None
    weights, chosen, offsets, rows, slots = s["routing"]
    cuts = offsets.tolist()
    e, t = case["experts"], case["tokens"]
    if op == "router":
        l = s["logits"].double()
        some = torch.isfinite(l).any(1)
        p = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], l, 0.0), dim=1), 0.0)
        f = torch.tensor([cuts[i + 1] - cuts[i] for i in range(e)], dtype=torch.float64, device="cuda") / cuts[-1]
        probs = p.sum(0) / some.sum()
        slope = s["coefficient"] * e * f / some.sum()
        loss = s["coefficient"] * e * (f * probs).sum()
        d = p * slope - p * (p @ slope)[:, None]
        q = torch.zeros(t, e + 1, dtype=torch.float64, device="cuda")  # the last column: no choice
        at = torch.where(chosen >= 0, chosen, e).long()
        q.scatter_(1, at, s["dweights"].double())
        picked = torch.zeros_like(q).scatter_(1, at, 1.0)[:, :e]
        w = p * picked
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
            d = d + w * (q[:, :e] - (w * q[:, :e]).sum(1, keepdim=True))
        else:
            d = d + w * q[:, :e] - p * (w * q[:, :e]).sum(1, keepdim=True)
        return loss, None, probs, d
    total = t * s["top_k"]
    if op == "experts":
        if 2 * total * case["n"] * case["k"] > 1e13:
            return None
        n = case["n"]
        a = _values64(s["a"], s["as"])
        out = torch.empty(total, n, dtype=torch.float64, device="cuda")
        for i in range(e):
            mine = slice(cuts[i], cuts[i + 1])
            w = s["w"][i * n:(i + 1) * n].double().view(n // 128, 128, -1, 128) * s["ws"][i * n // 128:(i + 1) * n // 128].double()[:, None, :, None]
            out[mine] = (a[rows[mine].long()] if case["gather"] else a[mine]) @ w.view(n, -1).T
        return out
    if op == "swiglu_grad":
        w = case["width"]
        v = _values64(s["saved"], s["saved_scales"])
        g, u, dy = v[:, :w], v[:, w:], s["dy"].double().clone()
        dy[cuts[-1]:] = 0
        sig = torch.sigmoid(g)
        dots = (dy * g * sig * u).sum(1)
        ok = slots >= 0
        weight = torch.zeros(total, dtype=torch.float64, device="cuda")
        weight[slots[ok].long()] = weights[ok].double()
        dots = torch.where(ok, dots[slots.clamp(min=0).long()], 0.0)
        dy *= weight[:, None]
        dx = torch.cat([dy * u * (sig + g * sig * (1 - sig)), dy * g * sig], dim=1)
        act = weight[:, None] * g * sig * u
        codes, scales = _over_scales64(dx, case["mode"])
        mine = [slice(cuts[i], cuts[i + 1]) for i in range(e)]
        cap = _capacity(total, e)
        return (codes, scales if case["mode"] == "fp8_block128" else None, dots, _as_images64([dx[m] for m in mine], cap), None,
                _as_images64([act[m] for m in mine], cap), None)
    if 2 * total * case["n"] * case["k"] > 1e13:
        return None
    # the layer's input is what its codes and scales stand for in 32 bits: with scales of amax / 448 many of
    # those values lie on the border between two codes of the columns
    x = s["x"].double() if s["xs"] is None else _values64(s["x"], s["xs"]).float().double()
    out = torch.zeros(e, case["n"], case["k"], dtype=torch.float64, device="cuda")
    for i in range(e):
        both = []
        for v in (s["dy"][cuts[i]:cuts[i + 1]].double(), x[rows[cuts[i]:cuts[i + 1]].long()]):
            v = torch.cat([v, v.new_zeros(-v.shape[0] % 32, v.shape[1])]).T.unflatten(1, (-1, 32))
            scale = torch.exp2(_block_exponent64(v))[:, :, None]
            both.append((_e4m3_64(v / scale) * scale).flatten(1))
        if both[0].shape[1]:
            out[i] = both[0] @ both[1].T
    return out
