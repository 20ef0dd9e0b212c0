"""Binding of the operators around the GEMM: quantisation of activations, RMS
norm with quantised output, and a mixture-of-experts layer's routing and
weighted sum.  Argument marshalling and checks only, as in the package's
``__init__``.

Calls of a few microseconds: checks are plain comparisons, and the stream is
read without making a Stream object.
"""
import ctypes
import functools
from typing import NamedTuple

import torch

import mx_gemm_gb300 as _fg

FG_TYPE_F32, FG_TYPE_BF16 = 0, 1
FG_ACT_NONE, FG_ACT_SWIGLU = 0, 1
FG_FLAG_RENORMALIZE = 0x1
_TYPES = {torch.float32: FG_TYPE_F32, torch.bfloat16: FG_TYPE_BF16}
_ACTS = {"none": FG_ACT_NONE, "swiglu": FG_ACT_SWIGLU}
_E4M3 = torch.float8_e4m3fn
_E8M0 = torch.float8_e8m0fnu
_raw_stream = torch._C._cuda_getCurrentRawStream


class Routing(NamedTuple):
    """What moe_route returns (see fg_moe_route in include/fg.h)."""
    weights: torch.Tensor   # fp32 [T][top_k]
    experts: torch.Tensor   # int32 [T][top_k]
    offsets: torch.Tensor   # int32 [E + 1]
    rows: torch.Tensor      # int32 [T * top_k]: token of each slot
    slots: torch.Tensor     # int32 [T][top_k]: slot of each choice


def _rows(t, name, device=None):
    """A 2-D CUDA tensor whose rows are contiguous (any distance apart): its (rows, columns, distance)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (it is on %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the other operands on %s" % (name, t.device, device))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    m, k = t.shape
    ld, inner = t.stride()
    if inner != 1 and k > 1:
        raise ValueError("%s must have contiguous rows (shape %s, strides %s)" % (name, tuple(t.shape), t.stride()))
    if m <= 1:  # the distance of a single row says nothing
        ld = max(k, 1)
    elif ld < k:
        raise ValueError("%s has overlapping rows (shape %s, strides %s)" % (name, tuple(t.shape), t.stride()))
    return m, k, ld


def _type(t, name):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError("%s has dtype %s; expected torch.float32 or torch.bfloat16" % (name, t.dtype)) from None


def _on(device, stream, *tensors):
    """The stream handle of a launch on `device`; tensors allocated here are
    kept from reuse until a stream other than the current one is done with them."""
    if device.index != torch._C._cuda_getDevice():
        raise ValueError("the operands are on %s, the current device is cuda:%d" % (device, torch._C._cuda_getDevice()))
    current = _raw_stream(device.index)
    if stream is None:
        return current
    handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if handle != current:
        other = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device)
        for t in tensors:
            if t is not None:
                t.record_stream(other)
    return handle


def _p(t):
    return None if t is None else t.data_ptr()


def _code_outputs(mode, m, k, device):
    """Empty codes and scales of an [m][k] operand."""
    if mode == _fg.FG_MXFP4:
        codes = torch.empty((m, k // 2), dtype=torch.uint8, device=device)
    else:
        codes = torch.empty((m, k), dtype=_E4M3, device=device)
    if mode == _fg.FG_FP8_BLOCK128:
        return codes, torch.empty((m, k // 128), dtype=torch.float32, device=device)
    return codes, torch.empty((m, k // (128 if mode == _fg.FG_MXFP8 else 32)), dtype=_E8M0, device=device)


def quantize(mode, x, act="none", stream=None):
    """(codes, scales) of the A operand of `mode` from x [M][K] (fp32 or bf16),
    or with act="swiglu" from rows (g, u) of 2K values.

    Codes are float8_e4m3fn [M][K] (uint8 [M][K/2], two e2m1 codes a byte, for
    mxfp4); scales float8_e8m0fnu [M][K/32] ([M][K/128] for mxfp8), or fp32
    [M][K/128] for fp8_block128.  The rows of x may be any distance apart.
    """
    mode = _fg._mode(mode)
    act = _ACTS[act] if act in _ACTS else int(act)
    m, k, ld = _rows(x, "x")
    if act == FG_ACT_SWIGLU:
        if k % 2:
            raise ValueError("x must have rows (g, u) of two equal halves, got %d columns" % k)
        k //= 2
    device = x.device
    codes, scales = _code_outputs(mode, m, k, device)
    _fg._check(_fg.lib().fg_quantize(mode, act, x.data_ptr(), _type(x, "x"), m, k, ld, codes.data_ptr(),
                                     scales.data_ptr(), _on(device, stream, codes, scales)))
    return codes, scales


def rmsnorm_quantize(mode, x, weight, residual=None, eps=1e-6, normed=False, stream=None):
    """(codes, scales, h, y) of y = RMSnorm(h) * weight with h = x + residual.

    codes and scales as quantize() gives them (None for mode "bf16"); h, the new
    residual, is None where no residual is given; y is None unless `normed` is
    set or the mode is "bf16".  x, residual and weight are all fp32 or all bf16,
    and so are h and y.
    """
    mode = _fg._mode(mode)
    m, k, ldx = _rows(x, "x")
    device, t = x.device, _type(x, "x")
    if not isinstance(weight, torch.Tensor) or weight.device != device or weight.dtype != x.dtype or \
            weight.shape != (k,) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous %s tensor of %d values on %s" % (x.dtype, k, device))
    ldr, h = k, None
    if residual is not None:
        mr, kr, ldr = _rows(residual, "residual", device)
        if (mr, kr) != (m, k) or residual.dtype != x.dtype:
            raise ValueError("residual must be %s of shape %s, got %s %s" % (x.dtype, (m, k), residual.dtype, (mr, kr)))
        h = torch.empty((m, k), dtype=x.dtype, device=device)
    plain = mode == _fg.FG_BF16
    codes, scales = (None, None) if plain else _code_outputs(mode, m, k, device)
    y = torch.empty((m, k), dtype=x.dtype, device=device) if plain or normed else None
    _fg._check(_fg.lib().fg_rmsnorm_quantize(mode, x.data_ptr(), ldx, _p(residual), ldr, weight.data_ptr(), eps, t, m, k,
                                             _p(h), _p(y), _p(codes), _p(scales), _on(device, stream, codes, scales, h, y)))
    return codes, scales, h, y


@functools.lru_cache(maxsize=4096)  # a call of its own costs as much as an allocation
def _route_workspace(device_index, tokens, experts):
    return moe_route_workspace_size(tokens, experts)


def moe_route_workspace_size(tokens, experts):
    b = ctypes.c_uint64()
    _fg._check(_fg.lib().fg_moe_route_workspace_size(tokens, experts, ctypes.byref(b)))
    return b.value


def moe_route(logits, top_k, renormalize=True, stream=None):
    """Routing of the tokens of logits [T][E] (fp32 or bf16) to top_k experts
    each: a Routing (weights, experts, offsets, rows, slots)."""
    t, e, ld = _rows(logits, "logits")
    device = logits.device
    top_k = int(top_k)
    if not 0 < top_k <= max(e, 1):
        raise ValueError("top_k=%d outside 1..%d" % (top_k, e))
    weights = torch.empty((t, top_k), dtype=torch.float32, device=device)
    experts = torch.empty((t, top_k), dtype=torch.int32, device=device)
    offsets = torch.empty(e + 1, dtype=torch.int32, device=device)
    rows = torch.empty(t * top_k, dtype=torch.int32, device=device)
    slots = torch.empty((t, top_k), dtype=torch.int32, device=device)
    need = _route_workspace(device.index, t, e)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _fg._check(_fg.lib().fg_moe_route(logits.data_ptr(), _type(logits, "logits"), t, e, ld, top_k,
                                      FG_FLAG_RENORMALIZE if renormalize else 0, weights.data_ptr(), experts.data_ptr(),
                                      offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), _p(ws), need,
                                      _on(device, stream, weights, experts, offsets, rows, slots, ws)))
    return Routing(weights, experts, offsets, rows, slots)


@functools.lru_cache(maxsize=4096)
def _grouped_workspace(device_index, mode, rows, experts, n, k, gather):
    return grouped_gemm_workspace_size(mode, rows, experts, n, k, gather)


def grouped_gemm_workspace_size(mode, rows, experts, n, k, gather=False):
    """Workspace bytes of grouped_gemm for `rows` rows of Y (gather: with row indexes)."""
    b = ctypes.c_uint64()
    _fg._check(_fg.lib().fg_grouped_gemm_workspace_size(_fg._mode(mode), rows, experts, n, k, int(gather), ctypes.byref(b)))
    return b.value


def grouped_gemm(A, pb, offsets, a_scales=None, rows=None, Y=None, workspace=None, flags=0, stream=None):
    """Y[i] = dequant(A[rows[i]]) . dequant(B_e)^T (bf16 [R][N]) for the rows i of
    expert e, offsets[e] <= i < offsets[e+1].

    pb is the preshuffled stack of the experts' weights, [E * N][K]; offsets is
    int32 [E + 1] on the device; A holds codes [T][K] as for gemm().  rows (int32
    [R]) names the row of A for each row of Y; without it they are the same.
    Rows of Y that no expert holds are left as they are.
    """
    mode, n_all, k = pb.mode, pb.N, pb.K
    device = pb.data.device
    _fg._require(A, "A", _fg._a_dtypes(mode), device)
    if A.dim() != 2 or _fg._row_bytes_of(A) != _fg._a_row_bytes(mode, k):
        raise ValueError("A must be [T][K] codes of the mode (%d bytes per row for K=%d), got shape %s dtype %s"
                         % (_fg._a_row_bytes(mode, k), k, tuple(A.shape), A.dtype))
    t = A.shape[0]
    _fg._require(offsets, "offsets", (torch.int32,), device)
    e = offsets.numel() - 1
    if e < 1 or n_all % e:
        raise ValueError("offsets must hold E + 1 values, E a divisor of the stacked weight's %d rows" % n_all)
    n = n_all // e
    if a_scales is not None and mode != _fg.FG_BF16:
        dts, count = _fg._scale_spec(mode, t, k, False)
        _fg._require(a_scales, "a_scales", dts, device, numel=count)
    if rows is not None:
        _fg._require(rows, "rows", (torch.int32,), device)
    r = t if rows is None else rows.numel()
    if Y is None:
        Y = torch.empty((r, n), dtype=torch.bfloat16, device=device)
    else:
        _fg._require(Y, "Y", _fg._dtypes("bfloat16", "int16"), device, shape=(r, n))
    need = 0
    if workspace is None:
        need = _grouped_workspace(device.index, mode, r, e, n, k, rows is not None)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _fg._require(workspace, "workspace", device=device)
        need = workspace.numel() * workspace.element_size()
    _fg._check(_fg.lib().fg_grouped_gemm(A.data_ptr(), _p(a_scales), t, _p(rows), r, offsets.data_ptr(), e,
                                         ctypes.byref(pb.desc), mode, Y.data_ptr(), _p(workspace), need, flags,
                                         _on(device, stream, Y, workspace)))
    return Y


def moe_combine(Y, slots, weights, residual=None, stream=None):
    """out[t] = residual[t] + sum_j weights[t][j] * Y[slots[t][j]] (bf16 [T][N])
    for the experts' rows Y [R][N]; a slot of -1 is no choice."""
    _fg._require(Y, "Y", (torch.bfloat16,))
    device = Y.device
    _fg._require(slots, "slots", (torch.int32,), device)
    if Y.dim() != 2 or slots.dim() != 2:
        raise ValueError("Y and slots must be 2-D, got shapes %s and %s" % (tuple(Y.shape), tuple(slots.shape)))
    t, k = slots.shape
    r, n = Y.shape
    _fg._require(weights, "weights", (torch.float32,), device, shape=(t, k))
    if residual is not None:
        _fg._require(residual, "residual", (torch.bfloat16,), device, shape=(t, n))
    out = torch.empty((t, n), dtype=torch.bfloat16, device=device)
    _fg._check(_fg.lib().fg_moe_combine(Y.data_ptr(), r, slots.data_ptr(), weights.data_ptr(), _p(residual), t, k, n,
                                        out.data_ptr(), _on(device, stream, out)))
    return out
