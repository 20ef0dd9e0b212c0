"""Host-side refusals of the operators around the GEMM (no GPU needed): every
bad argument is reported before anything is launched."""
import ctypes

import pytest
import torch

from tests.test_abi import fg  # noqa: F401  (fixture)

P = 1 << 20  # a well-aligned address that is never read


def ptr(x=P):
    return ctypes.c_void_p(x)


def quantize(fg, mode=5, act=0, x=P, type=1, M=4, K=256, ldx=None, codes=2 * P, scales=3 * P):
    return fg.lib().fg_quantize(mode, act, ptr(x), type, M, K, (2 * K if act == 1 else K) if ldx is None else ldx,
                                ptr(codes), ptr(scales), None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=0), "INVALID_ARG"), (dict(mode=1), "INVALID_ARG"), (dict(mode=7), "INVALID_ARG"), (dict(mode=-1), "INVALID_ARG"),
    (dict(act=2), "INVALID_ARG"), (dict(type=2), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(codes=0), "INVALID_ARG"),
    (dict(scales=0), "INVALID_ARG"), (dict(M=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=48), "SHAPE"),
    (dict(mode=3, K=96), "SHAPE"), (dict(mode=2, K=96), "SHAPE"), (dict(ldx=248), "SHAPE"), (dict(act=1, ldx=256), "SHAPE"),
    (dict(M=1 << 25), "SHAPE"), (dict(x=P + 8), "ALIGN"), (dict(ldx=257), "ALIGN"), (dict(codes=P + 8), "ALIGN"),
    (dict(mode=2, scales=P + 2), "ALIGN"),
])
def test_quantize_refusals(fg, bad, status):  # noqa: F811
    assert quantize(fg, **bad) == getattr(fg, "FG_ERR_" + status)
    assert "fg_quantize" in fg.last_error_message()


def norm(fg, mode=5, x=P, ldx=256, residual=2 * P, ldr=256, weight=3 * P, eps=1e-6, type=1, M=4, K=256, h=4 * P, y=5 * P,
         codes=6 * P, scales=7 * P):
    return fg.lib().fg_rmsnorm_quantize(mode, ptr(x), ldx, ptr(residual), ldr, ptr(weight), eps, type, M, K, ptr(h), ptr(y),
                                        ptr(codes), ptr(scales), None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=1), "INVALID_ARG"), (dict(mode=9), "INVALID_ARG"), (dict(type=5), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"),
    (dict(weight=0), "INVALID_ARG"), (dict(codes=0), "INVALID_ARG"), (dict(mode=0), "INVALID_ARG"),
    (dict(mode=0, codes=0, scales=0, y=0), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(K=48, ldx=48, ldr=48), "SHAPE"), (dict(K=65536, ldx=65536, ldr=65536), "SHAPE"), (dict(ldx=128), "SHAPE"),
    (dict(ldr=128), "SHAPE"), (dict(x=P + 2), "ALIGN"), (dict(residual=P + 8), "ALIGN"), (dict(weight=P + 8), "ALIGN"),
    (dict(h=P + 8), "ALIGN"), (dict(y=P + 8), "ALIGN"), (dict(ldr=260), "ALIGN"),
])
def test_norm_refusals(fg, bad, status):  # noqa: F811
    assert norm(fg, **bad) == getattr(fg, "FG_ERR_" + status)
    assert "fg_rmsnorm_quantize" in fg.last_error_message()


def route(fg, logits=P, type=0, T=100, E=64, ldl=64, k=4, flags=1, weights=2 * P, experts=3 * P, offsets=4 * P, rows=5 * P,
          slots=6 * P, ws=7 * P, bytes=1 << 20):
    return fg.lib().fg_moe_route(ptr(logits), type, T, E, ldl, k, flags, ptr(weights), ptr(experts), ptr(offsets), ptr(rows),
                                 ptr(slots), ptr(ws), bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(type=3), "INVALID_ARG"), (dict(flags=2), "INVALID_ARG"), (dict(logits=0), "INVALID_ARG"), (dict(offsets=0), "INVALID_ARG"),
    (dict(slots=0), "INVALID_ARG"), (dict(T=-1), "SHAPE"), (dict(E=0), "SHAPE"), (dict(E=1025, ldl=1025), "SHAPE"),
    (dict(k=0), "SHAPE"), (dict(k=33), "SHAPE"), (dict(E=3, k=4), "SHAPE"), (dict(ldl=63), "SHAPE"), (dict(T=1 << 29), "SHAPE"),
    (dict(logits=P + 2), "ALIGN"), (dict(rows=P + 2), "ALIGN"), (dict(ws=P + 4), "ALIGN"), (dict(ws=0), "WORKSPACE"),
    (dict(bytes=100), "WORKSPACE"),
])
def test_route_refusals(fg, bad, status):  # noqa: F811
    assert route(fg, **bad) == getattr(fg, "FG_ERR_" + status)
    assert "fg_moe_route" in fg.last_error_message()


def combine(fg, Y=P, R=64, slots=2 * P, weights=3 * P, residual=4 * P, T=8, k=8, N=256, out=5 * P):
    return fg.lib().fg_moe_combine(ptr(Y), R, ptr(slots), ptr(weights), ptr(residual), T, k, N, ptr(out), None)


@pytest.mark.parametrize("bad,status", [
    (dict(Y=0), "INVALID_ARG"), (dict(slots=0), "INVALID_ARG"), (dict(weights=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"),
    (dict(T=-1), "SHAPE"), (dict(R=-1), "SHAPE"), (dict(N=0), "SHAPE"), (dict(N=100), "SHAPE"), (dict(k=0), "SHAPE"),
    (dict(k=33), "SHAPE"), (dict(Y=P + 8), "ALIGN"), (dict(residual=P + 8), "ALIGN"), (dict(out=P + 2), "ALIGN"),
    (dict(weights=P + 2), "ALIGN"),
])
def test_combine_refusals(fg, bad, status):  # noqa: F811
    assert combine(fg, **bad) == getattr(fg, "FG_ERR_" + status)
    assert "fg_moe_combine" in fg.last_error_message()


def descriptor(fg, mode, N, K):
    """A descriptor with a valid check word (the buffers are never read)."""
    d = fg.BShuf()
    d.magic, d.version, d.mode, d.tile_rows, d.N, d.K = 0x31424746, 1, mode, 128, N, K
    d.data, d.sf, d.data_bytes, d.sf_bytes = 8 * P, 9 * P, N * K, N * K // 32
    h = 1469598103934665603
    for b in bytes(d)[:fg.BShuf.check.offset]:
        h = (h ^ b) * 1099511628211 % (1 << 64)
    d.check = h ^ 0x5eedf00dcafe1234
    return d


def grouped(fg, mode=5, dmode=None, N=8 * 256, K=512, A=P, a_scales=2 * P, T=40, rows=3 * P, R=80, offsets=4 * P, E=8, Y=5 * P,
            ws=6 * P, bytes=1 << 30, flags=0, desc=None):
    d = descriptor(fg, mode if dmode is None else dmode, N, K) if desc is None else desc
    return fg.lib().fg_grouped_gemm(ptr(A), ptr(a_scales), T, ptr(rows), R, ptr(offsets), E, ctypes.byref(d), mode, ptr(Y),
                                    ptr(ws), bytes, flags, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dmode=4), "LAYOUT"), (dict(mode=9, dmode=9), "INVALID_ARG"), (dict(mode=2, a_scales=P + 2), "ALIGN"), (dict(flags=1), "INVALID_ARG"), (dict(A=0), "INVALID_ARG"),
    (dict(Y=0), "INVALID_ARG"), (dict(offsets=0), "INVALID_ARG"), (dict(a_scales=0), "INVALID_ARG"),
    (dict(E=0), "SHAPE"), (dict(E=7), "SHAPE"), (dict(E=16, N=16 * 64), "SHAPE"), (dict(E=2048, N=2048 * 128), "SHAPE"),
    (dict(R=-1), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(T=0), "SHAPE"), (dict(rows=0), "SHAPE"), (dict(R=1 << 25), "SHAPE"),
    (dict(A=P + 8), "ALIGN"), (dict(Y=P + 8), "ALIGN"), (dict(rows=P + 2), "ALIGN"), (dict(offsets=P + 2), "ALIGN"),
    (dict(ws=P + 8), "ALIGN"), (dict(ws=0), "WORKSPACE"), (dict(bytes=64), "WORKSPACE"),
])
def test_grouped_refusals(fg, bad, status):  # noqa: F811
    assert grouped(fg, **bad) == getattr(fg, "FG_ERR_" + status), fg.last_error_message()


def test_grouped_refuses_a_descriptor_made_by_hand(fg):  # noqa: F811
    d = descriptor(fg, 5, 8 * 256, 512)
    d.N += 128 * 8
    assert grouped(fg, desc=d) == fg.FG_ERR_LAYOUT


def test_grouped_workspace_grows_with_what_is_laid_out(fg):  # noqa: F811
    size = fg.grouped_gemm_workspace_size
    assert size("mxfp8_b32", 0, 64, 4096, 7168) == 0
    assert size("bf16", 64 * 200, 64, 4096, 7168) == 0                       # many rows as they lie: nothing to lay out
    assert size("bf16", 64 * 200, 64, 4096, 7168, gather=True) == 64 * 200 * 7168 * 2
    assert size("mxfp4", 64 * 200, 64, 4096, 7168, gather=True) == (50 + 64) * 56 * 1024 + 64 * 200 * 3584
    assert size("mxfp8_b32", 64 * 40, 64, 4096, 7168) == (10 + 64) * 56 * 1024
    # few rows: two 32 x 128 fp32 partials and a ticket for each block
    few = size("mxfp8_b32", 64, 64, 4096, 7168)
    assert few > 0 and few % (2 * 32 * 128 * 4 + 8) == 0
    many = size("fp8_block128", 64 * 200, 64, 4096, 7168)                    # 32-row tiles whatever the rows
    assert many > 0 and many % (2 * 32 * 128 * 4 + 8) == 0


def test_no_rows_and_no_tokens_need_no_device(fg):  # noqa: F811
    assert grouped(fg, R=0) == fg.FG_OK
    assert quantize(fg, M=0) == fg.FG_OK and norm(fg, M=0) == fg.FG_OK and combine(fg, T=0) == fg.FG_OK


def test_off_arch_is_refused(fg):  # noqa: F811
    fg.debug_override_cc(9, 0)
    try:
        for call in (quantize, norm, route, combine, grouped):
            assert call(fg) in (fg.FG_ERR_UNSUPPORTED_ARCH, fg.FG_ERR_CUDA)  # (no device at all: CUDA)
    finally:
        fg.debug_override_cc(-1)


def test_binding_refuses_what_the_library_would_misread(fg):  # noqa: F811
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for call in (lambda: fg.quantize("mxfp4", x), lambda: fg.rmsnorm_quantize("bf16", x, x[0]),
                 lambda: fg.moe_route(x, 2), lambda: fg.moe_combine(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="Tensor"):
        fg.quantize("mxfp4", [1.0])
