"""Weights in 128 x 128 blocks, column operands, the gated activation's
checkpoint and the weights' gradients.

Where only rounding is done (weights, columns) codes and scales are compared for
equality with the 64-bit recipe.  The gradients' products: exact where every sum
is a whole number below 2^24; else within (slabs' MMAs + 32) * 2^-23 of the sum of
the products' magnitudes - each MMA rounds the sum once, and adds its 32 products
with no fewer bits than the largest has.
"""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def rand(seed, *shape, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    return x * torch.exp2(torch.randint(-6, 6, shape[:-1] + (1,), generator=g, device="cuda").float()) if spread else x


def same(a, b, what=""):
    assert torch.equal(a, b), "%s: %d of %d differ" % (what, int((a != b).sum()), a.numel())


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(128, 128), (128, 384), (640, 128), (3, 256, 384), (2, 384, 128)])
def test_weight(shape, dtype):
    w = rand(1, *shape).to(dtype)
    w.view(-1, shape[-2], shape[-1])[0, :128, :128] = 0          # a block of zeros: scale 1
    w.view(-1, shape[-2], shape[-1])[-1, -1, -1] = 100.0
    for transpose in (False, True):
        codes, scales = fg.quantize_weight("fp8_block128", w, transpose=transpose)
        v = w.double().view(-1, shape[-2], shape[-1])
        v = (v.transpose(1, 2) if transpose else v).reshape(-1, shape[-2] if transpose else shape[-1])
        b = v.view(v.shape[0] // 128, 128, -1, 128).transpose(1, 2).flatten(2)   # [rows / 128][cols / 128][128 * 128]
        top = b.abs().amax(2)
        s = torch.where(top == 0, torch.ones_like(top), ref.over_448(top))
        q = ref.to_e4m3((b.float() / s.float()[:, :, None]).double())
        q = q.unflatten(2, (128, 128)).transpose(1, 2).reshape(v.shape)
        same(scales.double(), s, "scales")
        same(codes.double(), q, "codes")


def test_weight_views_and_values_that_are_not_numbers():
    big = rand(2, 4, 300, 400).to(torch.bfloat16)
    w = big[1:3, 20:148, 8:264]                                    # rows 400 apart, experts 300 * 400
    same(fg.quantize_weight("fp8_block128", w)[0].double(), fg.quantize_weight("fp8_block128", w.contiguous())[0].double())
    w = rand(3, 256, 256)
    w[5, 7], w[200, 9], w[3, 255] = NAN, INF, 1e-44
    codes, scales = fg.quantize_weight("fp8_block128", w)
    assert torch.isnan(scales).tolist() == [[True, False], [True, False]]
    assert (codes.double()[:128, :128] == 0).all() and (codes.double()[128:, :128] == 0).all() and codes.double()[0, 128:].any()
    tiny = torch.zeros(128, 128, device="cuda")
    tiny[0, 0] = 1e-44                                             # amax / 448 would be zero
    codes, scales = fg.quantize_weight("fp8_block128", tiny)
    assert scales.item() > 0 and codes.double()[0, 0] > 0


def test_a_quantised_weight_and_its_transpose_multiply():
    """x W^T and dy W by the products that the layer calls, against the values that the codes stand for."""
    w = rand(4, 256, 384, spread=False) / 20
    for transpose in (False, True):
        codes, scales = fg.quantize_weight("fp8_block128", w, transpose=transpose)
        pb = fg.preshuffle_b("fp8_block128", codes, scales)
        a, a_s = fg.quantize("fp8_block128", rand(5, 40, codes.shape[1], spread=False))
        y = fg.gemm(a, pb, a_s).double()
        values = codes.double() * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        want = ref.decoded(a, a_s) @ values.T
        ref.within(y, want, 2.0 ** -8 * want.abs() + 1e-3 * want.abs().amax())


# ------------------------------------------------------------------ columns

CUTS = [
    ([1], 0, 1),                                   # one row
    ([0, 1, 0, 2], 0, 3),                          # experts without rows
    ([128, 256, 1, 127], 0, 512),                  # whole slabs and one short of them
    ([129, 33, 31, 32, 65], 0, 290),
    ([5, 0, 7], 3, 20),                            # rows before the first and behind the last expert
    ([0, 0], 0, 5),                                # nobody has a row
]


@pytest.mark.parametrize("counts,first,rows", CUTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_columns(counts, first, rows, dtype):
    x = rand(6, rows, 256).to(dtype)
    offsets = ref.fixed_offsets(counts, first)
    c = fg.quantize_columns(x, offsets)
    assert (c.N, c.K, c.rows, c.experts) == (256, ref.capacity(rows, len(counts)), rows, len(counts))
    codes, scales = ref.matrix(c)
    want, want_scales = ref.quantized(ref.by_place(x.double(), offsets.tolist(), rows), "mxfp8_b32")
    same(scales, want_scales, "scales")
    same(codes, want, "codes")
    plain, sf = fg.unshuffle_b(c)                   # the descriptor is one the library takes
    same(plain.view(torch.float8_e4m3fn).double(), want)
    same(sf.long(), want_scales)


@pytest.mark.parametrize("mode", ref.MODES)
def test_columns_of_a_checkpoint_gathered(mode):
    x = rand(7, 61, 384)
    codes, scales = fg.quantize(mode, x)
    r, _ = ref.routing(61, 9, 3, 8, padded=0.2, empty=(4,))
    c = fg.quantize_columns(codes, r.offsets, scales=scales, rows=r.rows)
    v = ref.decoded(codes, scales)[r.rows.clamp(min=0).long()]
    got, got_scales = ref.matrix(c)
    want, want_scales = ref.quantized(ref.by_place(v, r.offsets.tolist(), r.rows.numel()), "mxfp8_b32")
    same(got_scales, want_scales, "scales")
    same(got, want, "codes")
    same(c.data, fg.quantize_columns(codes.view(torch.uint8), r.offsets, scales=scales, rows=r.rows).data)


def test_columns_of_all_rows_and_of_none():
    x = rand(9, 200, 128).to(torch.bfloat16)
    same(fg.quantize_columns(x).data, fg.quantize_columns(x, ref.fixed_offsets([200])).data)
    none = fg.quantize_columns(x[:0], ref.fixed_offsets([0, 0, 0]))
    assert none.K == 128 and not none.data.any() and (none.sf == 127).all()


def test_columns_of_a_view_and_bad_offsets_and_rows():
    big = rand(10, 100, 640).to(torch.bfloat16)
    x = big[::2, 128:384]
    offsets = ref.fixed_offsets([20, 30])
    same(fg.quantize_columns(x, offsets).data, fg.quantize_columns(x.contiguous(), offsets).data)
    # offsets that leave 0..R or decrease count as the largest before them, rows are clamped
    for bad in ([-4, 30, 20, 70], [0, 60, -9, 50], [40, 10, 45, 45]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c = fg.quantize_columns(x, o)
        want, scales = ref.quantized(ref.by_place(x.double(), bad, 50), "mxfp8_b32")
        same(ref.matrix(c)[0], want)
        same(ref.matrix(c)[1], scales)
    rows = torch.tensor([0, -1, 49, 50, 1 << 30, 7], dtype=torch.int32, device="cuda")
    c = fg.quantize_columns(x, ref.fixed_offsets([4, 2]), rows=rows)
    want, _ = ref.quantized(ref.by_place(x.double()[rows.clamp(0, 49).long()], [0, 4, 6], 6), "mxfp8_b32")
    same(ref.matrix(c)[0], want)


def test_columns_with_values_that_are_not_numbers_stay_within_their_blocks():
    x = rand(11, 70, 128)
    x[3, 5], x[40, 6], x[65, 7] = NAN, INF, -INF
    x[10] = 0
    x[:, 9] = 0
    x[0:32, 11] = 1e-45                             # the smallest value there is
    x[33, 12] = 3e38
    c = fg.quantize_columns(x, ref.fixed_offsets([70]))
    want, scales = ref.quantized(ref.by_place(x.double(), [0, 70], 70), "mxfp8_b32")
    same(ref.matrix(c)[1], scales)
    same(ref.matrix(c)[0], want)
    assert (ref.matrix(c)[1] == 255).sum() == 3


@pytest.mark.parametrize("experts", [33, 100, 1024])
def test_columns_of_many_experts(experts):
    g = torch.Generator().manual_seed(experts)
    counts = torch.randint(0, 4, (experts,), generator=g).tolist()
    rows = sum(counts) + 5
    x = rand(12, rows, 128).to(torch.bfloat16)
    offsets = ref.fixed_offsets(counts, 2)
    c = fg.quantize_columns(x, offsets)
    want, scales = ref.quantized(ref.by_place(x.double(), offsets.tolist(), rows), "mxfp8_b32")
    same(ref.matrix(c)[0], want)
    same(ref.matrix(c)[1], scales)


# --------------------------------------------------------------- checkpoint

@pytest.mark.parametrize("mode", ref.MODES + ("mxfp4_fp8a",))
@pytest.mark.parametrize("rows,width", [(1, 128), (3, 384), (130, 2048), (1000, 256), (0, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_checkpoint(mode, rows, width, dtype):
    """The same codes and scales as two calls of the quantiser."""
    x = rand(13, rows, 2 * width).to(dtype)
    if rows > 2:
        x[1, 5], x[2, width + 3], x[0, :128] = NAN, INF, 0
    got = fg.swiglu_checkpoint(mode, x)
    for a, b in zip(got, fg.quantize(mode, x, act="swiglu") + fg.quantize(mode, x)):
        assert a.dtype == b.dtype and a.shape == b.shape
        same(a.view(torch.uint8) if a.dtype != torch.float32 else a.view(torch.int32),
             b.view(torch.uint8) if b.dtype != torch.float32 else b.view(torch.int32))


def test_checkpoint_of_a_view():
    big = rand(14, 40, 3 * 512).to(torch.bfloat16)
    x = big[::2, 256:1280]
    for a, b in zip(fg.swiglu_checkpoint("mxfp8_b32", x), fg.swiglu_checkpoint("mxfp8_b32", x.contiguous())):
        same(a.view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------------- weights' gradient

def wgrad_ref(a, b, offsets, rows):
    """fp64 [E][N][K] and the sums of the products' magnitudes, from what the operands hold."""
    x, y = ref.column_values(a), ref.column_values(b)
    cuts = ref.clean(offsets.tolist(), rows)
    out, mag, p = [], [], 0
    for lo, hi in zip(cuts, cuts[1:]):
        q = p + -(-(hi - lo) // 128) * 128
        out.append(x[:, p:q] @ y[:, p:q].T)
        mag.append(x[:, p:q].abs() @ y[:, p:q].abs().T)
        p = q
    return torch.stack(out), torch.stack(mag)


def whole(seed, rows, cols):
    """Small whole numbers: three bits, which eight hold whatever the scale."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-7, 8, (rows, cols), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("counts,first,rows", CUTS + [([700, 0, 300], 0, 1000), ([3] * 40, 0, 120)])
@pytest.mark.parametrize("n,k", [(128, 128), (256, 256), (384, 128), (128, 640), (640, 384)])
def test_wgrad_exact(counts, first, rows, n, k):
    offsets = ref.fixed_offsets(counts, first)
    a, b = fg.quantize_columns(whole(15, rows, n), offsets), fg.quantize_columns(whole(16, rows, k), offsets)
    want, _ = wgrad_ref(a, b, offsets, rows)
    got = fg.grouped_wgrad(a, b, offsets)
    assert got.dtype == torch.float32 and got.shape == (len(counts), n, k)
    same(got.double(), want)
    # and directly from the rows: small whole numbers lose nothing in eight bits
    x, y, cuts = whole(15, rows, n).double(), whole(16, rows, k).double(), ref.clean(offsets.tolist(), rows)
    same(got.double(), torch.stack([x[i:j].T @ y[i:j] for i, j in zip(cuts, cuts[1:])]))
    same(fg.grouped_wgrad(a, b, offsets, dtype=torch.bfloat16), want.to(torch.bfloat16))
    out = torch.full_like(got, 3.0)
    assert fg.grouped_wgrad(a, b, offsets, out=out, accumulate=True) is out
    same(out.double(), want + 3)
    out = torch.full_like(got, NAN)
    same(fg.grouped_wgrad(a, b, offsets, out=out).double(), want)
    assert fg.get_error() == fg.FG_OK


@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(1, 8, 2, 256, 128), (300, 16, 4, 512, 384), (2500, 5, 2, 384, 1024),
                                                     (4096, 3, 3, 256, 256)])
def test_wgrad_of_random_values(tokens, experts, top_k, n, k):
    r, _ = ref.routing(tokens, experts, top_k, 17, padded=0.1)
    rows = tokens * top_k
    a = fg.quantize_columns(rand(18, rows, n).to(torch.bfloat16), r.offsets)
    b = fg.quantize_columns(rand(19, tokens, k).to(torch.bfloat16), r.offsets, rows=r.rows)
    want, mag = wgrad_ref(a, b, r.offsets, rows)
    got = fg.grouped_wgrad(a, b, r.offsets)
    most = int((r.offsets[1:] - r.offsets[:-1]).max())
    bound = (most / 32 + 32) * 2.0 ** -23 * mag
    ref.within(got, want, bound)
    half = fg.grouped_wgrad(a, b, r.offsets, dtype=torch.bfloat16)
    ref.within(half, want, bound + 2.0 ** -8 * want.abs())
    same(got, fg.grouped_wgrad(a, b, r.offsets))   # the same bits each time


def test_wgrad_of_values_that_are_not_numbers():
    """They reach the rows and columns of their own block, and their own expert."""
    x, y = rand(20, 300, 256), rand(21, 300, 128)
    x[10, 5], y[200, 7] = NAN, INF
    offsets = ref.fixed_offsets([100, 0, 200])
    out = fg.grouped_wgrad(fg.quantize_columns(x, offsets), fg.quantize_columns(y, offsets), offsets)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 5, :] = True
    bad[2, :, 7] = True
    same(torch.isnan(out), bad)


def test_wgrad_refuses_operands_of_other_rows():
    x = rand(22, 200, 128)
    a, b = fg.quantize_columns(x, ref.fixed_offsets([100, 100])), fg.quantize_columns(x[:150], ref.fixed_offsets([100, 50]))
    with pytest.raises(ValueError, match="rows"):
        fg.grouped_wgrad(a, b, ref.fixed_offsets([100, 100]))
    with pytest.raises(ValueError, match="experts"):
        fg.grouped_wgrad(a, a, ref.fixed_offsets([200]))
    with pytest.raises(ValueError, match="out"):
        fg.grouped_wgrad(a, a, ref.fixed_offsets([100, 100]), accumulate=True)
    with pytest.raises(ValueError, match="dtype"):
        fg.grouped_wgrad(a, a, ref.fixed_offsets([100, 100]), dtype=torch.float16)
    with pytest.raises(ValueError, match="out has"):
        fg.grouped_wgrad(a, a, ref.fixed_offsets([100, 100]), out=torch.empty(2, 128, 64, device="cuda"))
    with pytest.raises(fg.FgError, match="fp32"):
        fg.grouped_wgrad(a, a, ref.fixed_offsets([100, 100]), out=torch.empty(2, 128, 128, device="cuda", dtype=torch.bfloat16),
                         accumulate=True, dtype=torch.bfloat16)
    moved = fg.quantize_columns(x, ref.fixed_offsets([100, 100]))
    moved.data = moved.data.clone()
    with pytest.raises(ValueError, match="descriptor"):
        fg.grouped_wgrad(moved, a, ref.fixed_offsets([100, 100]))


def test_wgrad_that_times_out_says_so_and_the_next_call_is_right():
    x = whole(23, 700, 512)
    offsets = ref.fixed_offsets([300, 0, 400])
    a = fg.quantize_columns(x, offsets)
    want = fg.grouped_wgrad(a, a, offsets)
    torch.cuda.synchronize()
    fg.set_wait_timeout_ns(20_000_000)
    try:
        fg.grouped_wgrad(a, a, offsets, flags=fg.FG_FLAG_DEBUG_STALL)
        assert fg.get_error() == fg.FG_ERR_TIMEOUT
    finally:
        fg.set_wait_timeout_ns(4_000_000_000)
    same(fg.grouped_wgrad(a, a, offsets), want)
    assert fg.get_error() == fg.FG_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [0, 30, -30, 110, -110])
def test_weight_quotients_are_those_of_the_division(dtype, size):
    """Sixteen million of them, bf16's among which are many next to a border between two codes; and sizes at both ends."""
    w = torch.ldexp(rand(24, 4096, 4096), torch.tensor(size, device="cuda")).to(dtype)
    codes, scales = fg.quantize_weight("fp8_block128", w)
    s = scales.repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = (w.float() / s).to(torch.float8_e4m3fn)               # (tensor by tensor: rounded once)
    same(codes.view(torch.uint8), want.view(torch.uint8))
    # and the row blocks of the gated activation's gradient
    x = w.float()[:512]
    saved, saved_scales = fg.quantize("fp8_block128", torch.cat([x * 0 + 88, x * 0 + 1], 1))
    d = fg.swiglu_backward("fp8_block128", x, saved, saved_scales, plain=True)
    s = d.scales.repeat_interleave(128, 1)
    same(d.codes.view(torch.uint8), (d.dx / s).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [0, 30, -30, 110, -110])
def test_row_quotients_are_those_of_the_division(dtype, size):
    """The same for rows' blocks, of the quantiser and of both halves of a checkpoint."""
    x = torch.ldexp(rand(25, 2048, 4096), torch.tensor(size, device="cuda")).to(dtype)
    codes, scales = fg.quantize("fp8_block128", x)
    _, _, saved, saved_scales = fg.swiglu_checkpoint("fp8_block128", x)
    top = x.float().view(2048, 32, 128).abs().amax(2)
    same(scales, torch.where(top == 0, torch.ones_like(top), ref.over_448(top).float()))
    want = (x.float() / scales.repeat_interleave(128, 1)).to(torch.float8_e4m3fn)
    same(codes.view(torch.uint8), want.view(torch.uint8))
    same(saved.view(torch.uint8), want.view(torch.uint8))
    same(saved_scales, scales)
