"""Plain 64-bit forms of the training operators, for the GPU tests."""
import torch

import mx_gemm_gb300 as fg

MODES = ("mxfp8_b32", "mxfp8", "fp8_block128")
BLOCK = {"mxfp8_b32": 32, "mxfp8": 128, "fp8_block128": 128}
REL = 2.0 ** -18   # of a value: at most 20 operations of 2^-24 and two fast functions of 2 ulp
HALF = 2.0 ** -4   # half a step of e4m3, relative; its smallest step is 2^-9


def to_e4m3(v):
    """Nearest e4m3 values of fp64 v, ties to even, saturated."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448)


def exponent(amax):
    """127 + the smallest whole e with amax <= 448 * 2^e, in 0..254; 127 for zero, 255 if not finite."""
    m, e = torch.frexp(amax)
    c = (127 + e.to(torch.int64) - 9 + (m > 0.875)).clamp(0, 254)
    c = torch.where(amax == 0, 127, c)
    return torch.where(torch.isfinite(amax), c, 255)


def over_448(amax):
    """amax / 448 rounded once to 32 bits (by a tensor: torch multiplies by a number's reciprocal)."""
    return (amax.float() / torch.full_like(amax, 448.0, dtype=torch.float32)).double()


def blocks(v, size):
    return v.unflatten(-1, (-1, size))


def quantized(v, mode):
    """(values of the codes, scales) of v [..][K] (fp64 holding 32-bit values) by the recipe."""
    b = blocks(v, BLOCK[mode])
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    b = torch.where(bad[..., None], 0.0, b)
    if mode == "fp8_block128":
        s = torch.where(amax == 0, 1.0, over_448(amax))
        q = (b.float() / s.float()[..., None]).double()
        return to_e4m3(q).flatten(-2), torch.where(bad, float("nan"), s)
    c = exponent(amax)
    return to_e4m3(b * torch.exp2(127.0 - torch.where(bad, 127, c))[..., None]).flatten(-2), c


def scale_values(scales):
    """fp64 values of E8M0 or fp32 scales."""
    if scales.dtype == torch.float32:
        return scales.double()
    c = scales.view(torch.uint8).double()
    return torch.where(c == 255, float("nan"), torch.exp2(c - 127))


def decoded(codes, scales):
    """fp64 values that codes and scales stand for, rounded to 32 bits."""
    s = scale_values(scales).view(codes.shape[0], -1)
    return (codes.view(torch.float8_e4m3fn).double() * s.repeat_interleave(codes.shape[1] // s.shape[1], 1)).float().double()


def capacity(rows, experts):
    return 128 * max(1, rows // 128 + min(experts, rows))


def clean(offsets, rows):
    """Offsets as the operators read them: clamped, each at least the one before."""
    out = []
    for o in offsets:
        o = min(max(int(o), 0), rows)
        out.append(max(o, out[-1]) if out else o)
    return out


def places(offsets, rows):
    """Row of each place of a column operand, -1 where there is none."""
    cuts = clean(offsets, rows)
    at = torch.full((capacity(rows, len(cuts) - 1),), -1, dtype=torch.int64)
    p = 0
    for a, b in zip(cuts, cuts[1:]):
        at[p:p + b - a] = torch.arange(a, b)
        p += -(-(b - a) // 128) * 128
    return at


def by_place(v, offsets, rows):
    """v's rows [rows][C] as columns [C][P], zeros where there is no row."""
    at = places(offsets, rows).to(v.device)
    if rows == 0:
        return v.new_zeros(v.shape[1], at.numel())
    return torch.where(at[:, None] >= 0, v[at.clamp(min=0)], 0.0).T.contiguous()


def matrix(c):
    """(fp64 values of the codes [C][P], E8M0 codes [C][P / 32]) of a column operand, by the layout's definition."""
    n, p = c.N, c.K
    b = c.data.view(n // 128, p // 128, 128, 8, 16)
    r = torch.arange(128, device=b.device)[:, None]
    piece = torch.arange(8, device=b.device)[None, :] ^ (r % 8)
    codes = b[:, :, r, piece].reshape(n // 128, p // 128, 128, 128).transpose(1, 2).reshape(n, p)
    atoms = c.sf.view(n // 128, p // 128, 32, 4, 4)      # [row % 32][row / 32][32 places]
    scales = atoms.permute(0, 3, 2, 1, 4).reshape(n, p // 32)
    return codes.contiguous().view(torch.float8_e4m3fn).double(), scales.long()


def column_values(c):
    """fp64 values that a column operand stands for, [C][P]."""
    codes, scales = matrix(c)
    s = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return codes * s.repeat_interleave(32, 1)


def within(got, want, bound, what=""):
    """|got - want| <= bound everywhere, or the worst place is named."""
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = int(((got - want).abs() / bound.clamp(min=1e-300)).nan_to_num(nan=float("inf"), posinf=1e300).flatten().argmax())
        raise AssertionError("%s: %d of %d off, the worst at %d of %s: %.9g for %.9g, bound %.3g"
                             % (what, int(bad.sum()), bad.numel(), i, tuple(got.shape), got.flatten()[i], want.flatten()[i],
                                bound.flatten()[i]))


def near(codes, scales, ref, mag, mode, what=""):
    """Codes (fp64 values) and scales against 64-bit values `ref` whose 32-bit
    arithmetic is off by at most REL * mag: each value within half a step, each
    scale that of a maximum within the arithmetic's error of the block's."""
    size = BLOCK[mode] if mode in BLOCK else 32
    r, m = blocks(ref, size), blocks(mag, size)
    s = scale_values(scales) if scales.dtype in (torch.float32, torch.uint8, torch.float8_e8m0fnu) else torch.exp2(scales.double() - 127)
    s = s.view(r.shape[:-1])
    off = REL * m
    lo, hi = (r.abs() - off).amax(-1).clamp(min=0), (r.abs() + off).amax(-1)
    if mode == "fp8_block128":
        ok = (s >= lo / 448 * (1 - 2.0 ** -23)) & (s <= hi / 448 * (1 + 2.0 ** -23))
        ok |= (hi < 2.0 ** -120) | (lo == 0) & ((s <= hi / 448 * (1 + 2.0 ** -23)) | (s == 1))  # (below 2^-132 s is rounded up)
    else:
        c = (torch.log2(s) + 127).round().long()
        # an interval down to 0 holds every smaller magnitude, and 0 itself (127)
        ok = (c <= exponent(hi)) & ((lo == 0) | (c >= exponent(lo))) | (lo == 0) & (c == 127)
    assert ok.all(), "%s: %d of %d scales off" % (what, int((~ok).sum()), ok.numel())
    v = blocks(codes, size) * s[..., None]
    bound = HALF * (1 + 2.0 ** -20) * r.abs() + 2.0 ** -10 * s[..., None] + 2 * off
    within(v, r, bound, what)


def routing(tokens, experts, top_k, seed, padded=0.0, empty=()):
    """moe_route()'s result for random logits, `empty` experts picked by nobody."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    logits[:, list(empty)] = -float("inf")
    logits[torch.rand(tokens, generator=g, device="cuda") < padded] = -float("inf")
    return fg.moe_route(logits, top_k), logits


def fixed_offsets(counts, first=0):
    out = [first]
    for c in counts:
        out.append(out[-1] + c)
    return torch.tensor(out, dtype=torch.int32, device="cuda")
