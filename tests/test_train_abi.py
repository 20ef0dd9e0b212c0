"""Host-side refusals of the training operators (no GPU needed): every bad
argument is reported before anything is launched."""
import ctypes

import pytest
import torch

from tests.test_abi import fg  # noqa: F401  (fixture)
from tests.test_moe_abi import P, descriptor, ptr


def weight(fg, mode=2, w=P, type=1, E=2, N=256, K=384, ldw=None, stride=None, transpose=0, codes=2 * P, scales=3 * P):
    ldw = K if ldw is None else ldw
    return fg.lib().fg_quantize_weight(mode, ptr(w), type, E, N, K, ldw, N * ldw if stride is None else stride, transpose,
                                       ptr(codes), ptr(scales), None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=5), "INVALID_ARG"), (dict(mode=0), "INVALID_ARG"), (dict(mode=9), "INVALID_ARG"), (dict(type=2), "INVALID_ARG"),
    (dict(w=0), "INVALID_ARG"), (dict(codes=0), "INVALID_ARG"), (dict(scales=0), "INVALID_ARG"), (dict(E=0), "SHAPE"),
    (dict(E=1025), "SHAPE"), (dict(N=0), "SHAPE"), (dict(N=64), "SHAPE"), (dict(K=192), "SHAPE"), (dict(K=1 << 21), "SHAPE"),
    (dict(ldw=256), "SHAPE"), (dict(w=P + 8), "ALIGN"), (dict(ldw=385), "ALIGN"), (dict(stride=9), "ALIGN"),
    (dict(stride=-8), "ALIGN"), (dict(codes=P + 8), "ALIGN"), (dict(scales=P + 2), "ALIGN"),
])
def test_weight_refusals(fg, bad, status):  # noqa: F811
    assert weight(fg, **bad) == getattr(fg, "FG_ERR_" + status)
    assert "fg_quantize_weight" in fg.last_error_message()


def checkpoint(fg, mode=5, x=P, type=1, M=4, K=256, ldx=None, codes=2 * P, scales=3 * P, saved=4 * P, saved_scales=5 * P):
    return fg.lib().fg_swiglu_checkpoint(mode, ptr(x), type, M, K, 2 * K if ldx is None else ldx, ptr(codes), ptr(scales),
                                         ptr(saved), ptr(saved_scales), None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=0), "INVALID_ARG"), (dict(mode=1), "INVALID_ARG"), (dict(mode=4), "INVALID_ARG"), (dict(mode=7), "INVALID_ARG"),
    (dict(type=2), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(codes=0), "INVALID_ARG"), (dict(saved=0), "INVALID_ARG"),
    (dict(saved_scales=0), "INVALID_ARG"), (dict(M=-1), "SHAPE"), (dict(K=48), "SHAPE"), (dict(mode=2, K=96), "SHAPE"),
    (dict(ldx=256), "SHAPE"), (dict(x=P + 8), "ALIGN"), (dict(ldx=513), "ALIGN"), (dict(saved=P + 8), "ALIGN"),
    (dict(mode=2, saved_scales=P + 2), "ALIGN"),
])
def test_checkpoint_refusals(fg, bad, status):  # noqa: F811
    assert checkpoint(fg, **bad) == getattr(fg, "FG_ERR_" + status)
    assert "fg_swiglu_checkpoint" in fg.last_error_message()


def columns(fg, mode=0, x=P, scales=0, type=1, T=40, C=256, ldx=256, rows=2 * P, R=80, offsets=3 * P, E=8, data=4 * P, sf=5 * P,
            desc=None):
    d = fg.BShuf()
    return fg.lib().fg_quantize_columns(mode, ptr(x), ptr(scales), type, T, C, ldx, ptr(rows), R, ptr(offsets), E, ptr(data),
                                        ptr(sf), ctypes.byref(d) if desc is None else None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=1), "INVALID_ARG"), (dict(mode=4), "INVALID_ARG"), (dict(mode=8), "INVALID_ARG"), (dict(type=4), "INVALID_ARG"),
    (dict(x=0), "INVALID_ARG"), (dict(scales=P), "INVALID_ARG"), (dict(mode=5), "INVALID_ARG"), (dict(offsets=0), "INVALID_ARG"),
    (dict(data=0), "INVALID_ARG"), (dict(sf=0), "INVALID_ARG"), (dict(desc=0), "INVALID_ARG"), (dict(E=0), "SHAPE"),
    (dict(E=1025), "SHAPE"), (dict(C=192, ldx=192), "SHAPE"), (dict(C=0), "SHAPE"), (dict(R=-1), "SHAPE"), (dict(T=0), "SHAPE"),
    (dict(T=-1), "SHAPE"), (dict(rows=0), "SHAPE"), (dict(R=1 << 21), "SHAPE"), (dict(ldx=128), "SHAPE"),
    (dict(mode=5, scales=P, ldx=512), "SHAPE"), (dict(x=P + 8), "ALIGN"), (dict(ldx=257), "ALIGN"), (dict(rows=P + 2), "ALIGN"),
    (dict(offsets=P + 2), "ALIGN"), (dict(data=P + 64), "ALIGN"), (dict(sf=P + 8), "ALIGN"),
    (dict(mode=2, scales=P + 2), "ALIGN"),
])
def test_columns_refusals(fg, bad, status):  # noqa: F811
    assert columns(fg, **bad) == getattr(fg, "FG_ERR_" + status), fg.last_error_message()
    assert "fg_quantize_columns" in fg.last_error_message()


def test_columns_sizes(fg):  # noqa: F811
    """128 places for every 128 rows and for every expert that can have one, at least 128."""
    assert fg.columns_size(256, 0, 8) == (128, 256 * 128, 256 * 4)
    assert fg.columns_size(256, 3, 8) == (3 * 128, 256 * 384, 256 * 12)
    assert fg.columns_size(128, 1000, 8) == ((7 + 8) * 128, 128 * 1920, 128 * 60)
    most = (1 << 20) - 8 * 128
    assert fg.columns_size(128, most, 8)[0] == 1 << 20
    with pytest.raises(fg.FgError, match="places"):
        fg.columns_size(128, most + 128, 8)


def backward(fg, mode=5, dy=P, type=1, R=80, K=256, ldd=256, saved=2 * P, saved_scales=3 * P, weights=4 * P, rows=5 * P,
             slots=6 * P, T=10, k=8, offsets=7 * P, E=8, codes=8 * P, scales=9 * P, dx=0, dweights=10 * P, dxd=11 * P, dxs=12 * P,
             ad=13 * P, asf=14 * P, ws=15 * P, bytes=1 << 20, descs=True):
    d = [ctypes.byref(fg.BShuf()) if descs else None for _ in range(2)]
    return fg.lib().fg_swiglu_backward(mode, ptr(dy), type, R, K, ldd, ptr(saved), ptr(saved_scales), ptr(weights), ptr(rows),
                                       ptr(slots), T, k, ptr(offsets), E, ptr(codes), ptr(scales), ptr(dx), ptr(dweights),
                                       ptr(dxd), ptr(dxs), d[0], ptr(ad), ptr(asf), d[1], ptr(ws), bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=0), "INVALID_ARG"), (dict(mode=4), "INVALID_ARG"), (dict(type=2), "INVALID_ARG"), (dict(dy=0), "INVALID_ARG"),
    (dict(saved=0), "INVALID_ARG"), (dict(codes=0), "INVALID_ARG"), (dict(scales=0), "INVALID_ARG"), (dict(rows=0), "INVALID_ARG"),
    (dict(slots=0), "INVALID_ARG"), (dict(dweights=0), "INVALID_ARG"), (dict(weights=0), "INVALID_ARG"),
    (dict(offsets=0), "INVALID_ARG"), (dict(dxd=0), "INVALID_ARG"), (dict(asf=0), "INVALID_ARG"), (dict(descs=False), "INVALID_ARG"),
    (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"), (dict(R=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=48, ldd=48), "SHAPE"),
    (dict(K=160, ldd=160), "SHAPE"), (dict(mode=2, K=96, ldd=96, dxd=0, dxs=0, ad=0, asf=0), "SHAPE"), (dict(ldd=128), "SHAPE"),
    (dict(k=0), "SHAPE"), (dict(k=33), "SHAPE"), (dict(T=0), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(R=1 << 21), "SHAPE"),
    (dict(dy=P + 8), "ALIGN"), (dict(ldd=257), "ALIGN"), (dict(saved=P + 8), "ALIGN"), (dict(codes=P + 8), "ALIGN"),
    (dict(dx=P + 8), "ALIGN"), (dict(weights=P + 2), "ALIGN"), (dict(offsets=P + 2), "ALIGN"), (dict(dxd=P + 64), "ALIGN"),
    (dict(ws=P + 2), "ALIGN"), (dict(ws=0), "WORKSPACE"), (dict(bytes=64), "WORKSPACE"),
])
def test_backward_refusals(fg, bad, status):  # noqa: F811
    assert backward(fg, **bad) == getattr(fg, "FG_ERR_" + status), fg.last_error_message()
    assert "fg_swiglu_backward" in fg.last_error_message()


def places(fg, R, E):
    return fg.columns_size(128, R, E)[0]


def wgrad(fg, N=256, K=384, R=80, E=8, pa=None, pb=None, offsets=P, type=0, accumulate=0, out=2 * P, flags=0, mode=5, desc=None):
    n = places(fg, 80, 8)
    a = descriptor(fg, mode, N, n if pa is None else pa) if desc is None else desc
    b = descriptor(fg, 5, K, n if pb is None else pb)
    return fg.lib().fg_grouped_wgrad(ctypes.byref(a), ctypes.byref(b), ptr(offsets), R, E, type, accumulate, ptr(out), flags, None)


@pytest.mark.parametrize("bad,status", [
    (dict(mode=2), "LAYOUT"), (dict(flags=1), "INVALID_ARG"), (dict(type=3), "INVALID_ARG"), (dict(type=1, accumulate=1), "INVALID_ARG"),
    (dict(offsets=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"), (dict(E=0), "SHAPE"), (dict(E=9), "SHAPE"),
    (dict(R=200), "SHAPE"), (dict(R=-1), "SHAPE"), (dict(pa=128), "SHAPE"), (dict(pb=128), "SHAPE"), (dict(offsets=P + 2), "ALIGN"),
    (dict(out=P + 8), "ALIGN"), (dict(N=1 << 24, K=1 << 24), "SHAPE"),
])
def test_wgrad_refusals(fg, bad, status):  # noqa: F811
    assert wgrad(fg, **bad) == getattr(fg, "FG_ERR_" + status), fg.last_error_message()


def test_wgrad_refuses_a_descriptor_made_by_hand(fg):  # noqa: F811
    d = descriptor(fg, 5, 256, places(fg, 80, 8))
    d.N += 128
    assert wgrad(fg, desc=d) == fg.FG_ERR_LAYOUT


def balance(fg, logits=P, type=0, T=1000, E=64, ldl=64, offsets=2 * P, c=0.01, loss=3 * P, counts=4 * P, probs=5 * P,
            slopes=6 * P, ws=7 * P, bytes=1 << 20):
    return fg.lib().fg_moe_balance_loss(ptr(logits), type, T, E, ldl, ptr(offsets), c, ptr(loss), ptr(counts), ptr(probs),
                                        ptr(slopes), ptr(ws), bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(type=3), "INVALID_ARG"), (dict(logits=0), "INVALID_ARG"), (dict(offsets=0), "INVALID_ARG"), (dict(loss=0), "INVALID_ARG"),
    (dict(counts=0), "INVALID_ARG"), (dict(probs=0), "INVALID_ARG"), (dict(slopes=0), "INVALID_ARG"), (dict(T=-1), "SHAPE"),
    (dict(T=1 << 25), "SHAPE"), (dict(E=0), "SHAPE"), (dict(E=1025, ldl=1025), "SHAPE"), (dict(ldl=63), "SHAPE"),
    (dict(logits=P + 2), "ALIGN"), (dict(offsets=P + 2), "ALIGN"), (dict(loss=P + 2), "ALIGN"), (dict(ws=P + 2), "ALIGN"),
    (dict(ws=0), "WORKSPACE"), (dict(bytes=100), "WORKSPACE"),
])
def test_balance_refusals(fg, bad, status):  # noqa: F811
    assert balance(fg, **bad) == getattr(fg, "FG_ERR_" + status), fg.last_error_message()
    assert "fg_moe_balance_loss" in fg.last_error_message()


def route_backward(fg, logits=P, type=0, T=100, E=64, ldl=64, experts=2 * P, dweights=3 * P, k=4, slopes=4 * P, flags=1, out=5 * P):
    return fg.lib().fg_moe_route_backward(ptr(logits), type, T, E, ldl, ptr(experts), ptr(dweights), k, ptr(slopes), flags, ptr(out),
                                          None)


@pytest.mark.parametrize("bad,status", [
    (dict(type=3), "INVALID_ARG"), (dict(flags=2), "INVALID_ARG"), (dict(logits=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"),
    (dict(experts=0), "INVALID_ARG"), (dict(T=-1), "SHAPE"), (dict(E=0), "SHAPE"), (dict(E=1025, ldl=1025), "SHAPE"),
    (dict(k=0), "SHAPE"), (dict(k=33), "SHAPE"), (dict(E=3, ldl=3, k=4), "SHAPE"), (dict(ldl=63), "SHAPE"),
    (dict(logits=P + 2), "ALIGN"), (dict(out=P + 2), "ALIGN"), (dict(slopes=P + 2), "ALIGN"), (dict(dweights=P + 2), "ALIGN"),
])
def test_route_backward_refusals(fg, bad, status):  # noqa: F811
    assert route_backward(fg, **bad) == getattr(fg, "FG_ERR_" + status), fg.last_error_message()
    assert "fg_moe_route_backward" in fg.last_error_message()


def test_no_rows_and_no_tokens_need_no_device(fg):  # noqa: F811
    assert checkpoint(fg, M=0) == fg.FG_OK and route_backward(fg, T=0) == fg.FG_OK
    assert backward(fg, R=0, weights=0, rows=0, slots=0, dweights=0, dxd=0, dxs=0, ad=0, asf=0) == fg.FG_OK


def test_off_arch_is_refused(fg):  # noqa: F811
    fg.debug_override_cc(9, 0)
    try:
        for call in (weight, checkpoint, columns, backward, wgrad, balance, route_backward):
            assert call(fg) in (fg.FG_ERR_UNSUPPORTED_ARCH, fg.FG_ERR_CUDA)  # (no device at all: CUDA)
    finally:
        fg.debug_override_cc(-1)


def test_binding_refuses_what_the_library_would_misread(fg):  # noqa: F811
    x = torch.zeros(128, 256, dtype=torch.bfloat16)
    for call in (lambda: fg.quantize_weight("fp8_block128", x), lambda: fg.swiglu_checkpoint("mxfp8", x),
                 lambda: fg.quantize_columns(x), lambda: fg.swiglu_backward("mxfp8", x, x, x),
                 lambda: fg.moe_balance_loss(x, x), lambda: fg.moe_route_backward(x, (x, x))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="column operand"):
        fg.grouped_wgrad(x, x, x)
    with pytest.raises(ValueError, match="8-bit"):
        fg.swiglu_checkpoint("mxfp4", x)
    with pytest.raises(ValueError, match="8-bit"):
        fg.swiglu_backward("bf16", x, x, x)
