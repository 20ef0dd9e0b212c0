"""Operators that train a mixture-of-experts layer in 8 bits: the weights' 128 x
128 blocks, the gated activation with its checkpoint and backward pass, the
weights' gradients, and the router's balance loss and gradient.

They are called as those of ``moe.py`` are (the compiled binding, streams,
errors); ``include/fg.h`` has the formulas.  An input's gradient is
``grouped_gemm`` with the transposed weight.  Gradients are calls, not autograd
nodes, and nothing waits for the device, so that a whole training step can be
captured in a CUDA graph.

Outputs that go together (codes and their scales, a column operand's two images, a
Balance's tensors) share one allocation: keeping one of them keeps the others' memory,
and saving one writes it too.  clone() what is kept or saved by itself.
"""
import ctypes
from typing import NamedTuple, Optional

import torch

import mx_gemm_gb300 as _fg
from mx_gemm_gb300 import moe

_TYPES = {torch.float32: moe.FG_TYPE_F32, torch.bfloat16: moe.FG_TYPE_BF16}


def _binding():
    return moe._binding or moe.binding()


class Columns(_fg.PreshuffledB):
    """A column operand of `rows` rows of `experts` experts: the image and scale
    image of an mxfp8_b32 matrix [N][K] with N columns and K places (see
    fg_columns_size in include/fg.h); unshuffle_b() gives the plain matrix."""

    def __init__(self, parts, rows, experts):
        data, sf, desc = parts
        super().__init__(_fg.BShuf.from_buffer_copy(desc), data, sf)
        self.rows, self.experts = rows, experts


class SwigluGrad(NamedTuple):
    """What swiglu_backward returns (see fg_swiglu_backward in include/fg.h)."""
    codes: torch.Tensor                   # e4m3 [R][2 K]: (dg, du)
    scales: torch.Tensor                  # as quantize() gives them
    dx: Optional[torch.Tensor]            # [R][2 K] in dy's type
    dweights: Optional[torch.Tensor]      # fp32 [T][top_k]
    dx_columns: Optional[Columns]         # 2 K columns
    act_columns: Optional[Columns]        # K columns: routing weight * activation


class Balance(NamedTuple):
    """What moe_balance_loss returns."""
    loss: torch.Tensor    # fp32 []
    counts: torch.Tensor  # int32 [E]: choices of each expert
    probs: torch.Tensor   # fp32 [E]: mean probability of each expert
    slopes: torch.Tensor  # fp32 [E]: the loss's derivative by each token's probability


def quantize_weight(mode, w, transpose=False, stream=None):
    """(codes, scales) of weights w [N][K] or [E][N][K] (fp32 or bf16) in the 128 x
    128 blocks of mode "fp8_block128", ready for preshuffle_b(): codes [E * N][K],
    or of the transposed weights [E * K][N].  The other modes' weights quantise row
    by row, with quantize()."""
    return _binding().quantize_weight(_fg._mode(mode), w, transpose, moe._handle(stream))


def swiglu_checkpoint(mode, x, stream=None):
    """(codes, scales, saved, saved_scales): quantize(mode, x, act="swiglu") and,
    from the same pass over x, quantize(mode, x), the checkpoint that
    swiglu_backward() takes.  mode: an 8-bit one."""
    return _binding().swiglu_checkpoint(_fg._mode(mode), x, moe._handle(stream))


def swiglu_backward(mode, dy, saved, saved_scales, routing=None, columns=False, plain=False, stream=None):
    """Gradients of the gated activation from its checkpoint: a SwigluGrad.

    dy [R][K] (fp32 or bf16) is the gradient of the activation's rows before their
    routing weight; routing is moe_route()'s result, whose weights the rows are
    multiplied by and whose rows of no expert are zero (None: no weights, all rows
    of one expert).  columns: the operands of grouped_wgrad() too; plain: (dg, du)
    in dy's type too.
    """
    r = routing if routing is not None else (None,) * 5
    codes, scales, dx, dweights, of_dx, of_act, rows, experts = _binding().swiglu_backward(
        _fg._mode(mode), dy, saved, saved_scales, r[0], r[3], r[4], r[2], columns, plain, moe._handle(stream))
    return SwigluGrad(codes, scales, dx, dweights, Columns(of_dx, rows, experts) if columns else None,
                      Columns(of_act, rows, experts) if columns else None)


def columns_size(columns, rows, experts):
    """(places, image bytes, scale image bytes) of a column operand."""
    p, d, s = ctypes.c_int64(), ctypes.c_uint64(), ctypes.c_uint64()
    _fg._check(_fg.lib().fg_columns_size(columns, rows, experts, ctypes.byref(p), ctypes.byref(d), ctypes.byref(s)))
    return p.value, d.value, s.value


def quantize_columns(x, offsets=None, scales=None, rows=None, stream=None):
    """Column operand (Columns) of the rows of x [T][C], fp32 or bf16, or e4m3 codes
    with `scales` as quantize() gives them in an 8-bit mode.

    offsets (int32 [E + 1]) divides the rows among the experts (None: one has them
    all); rows (int32 [R]) names the row of x for each (None: they are x's).
    """
    return Columns(*_binding().quantize_columns(x, offsets, scales, rows, moe._handle(stream)))


def grouped_wgrad(a, b, offsets, out=None, accumulate=False, dtype=torch.float32, flags=0, stream=None):
    """out[e] (fp32 or bf16 [E][N][K]) = the sum over the rows of expert e of a's row
    (N columns) times b's (K columns): the weights' gradient, for a from the
    gradients of a product's rows and b from its inputs, both column operands of
    the same offsets.  accumulate: `out` (fp32) is added to.
    """
    for name, t in (("a", a), ("b", b)):
        if not isinstance(t, Columns):
            raise ValueError("%s must be a column operand (quantize_columns), got %s" % (name, type(t).__name__))
    if (a.rows, a.experts) != (b.rows, b.experts):
        raise ValueError("a holds %d rows of %d experts, b %d of %d" % (a.rows, a.experts, b.rows, b.experts))
    if dtype not in _TYPES:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16, got %s" % dtype)
    return _binding().grouped_wgrad(a.data, a.sf, ctypes.addressof(a.desc), b.data, b.sf, ctypes.addressof(b.desc), offsets,
                                    a.rows, a.experts, out, accumulate, _TYPES[dtype], flags, moe._handle(stream))


def swiglu_backward_workspace_size(rows, width, weighted):
    b = ctypes.c_uint64()
    _fg._check(_fg.lib().fg_swiglu_backward_workspace_size(rows, width, int(weighted), ctypes.byref(b)))
    return b.value


def moe_balance_loss_workspace_size(tokens, experts):
    b = ctypes.c_uint64()
    _fg._check(_fg.lib().fg_moe_balance_loss_workspace_size(tokens, experts, ctypes.byref(b)))
    return b.value


def moe_balance_loss(logits, offsets, coefficient=0.01, stream=None):
    """Balance loss of the routing of logits [T][E] (fp32 or bf16) with the offsets
    (int32 [E + 1]) that moe_route() gave: a Balance (loss, counts, probs, slopes)."""
    return tuple.__new__(Balance, _binding().moe_balance_loss(logits, offsets, coefficient, moe._handle(stream)))


def moe_route_backward(logits, routing, dweights=None, slopes=None, renormalize=True, stream=None):
    """Gradient of logits [T][E], in their type, from that of the routing weights
    (dweights, fp32 [T][top_k]) and the slopes of the balance loss, each where
    given.  routing, renormalize: of the moe_route() call."""
    return _binding().moe_route_backward(logits, routing[1], dweights, slopes, renormalize, moe._handle(stream))
