"""Operators around the GEMM: quantisation of activations, RMS norm with
quantised output, and a mixture-of-experts layer's routing, grouped products
and weighted sum.

The functions check their tensors, allocate their outputs and call the C ABI
(``include/fg.h`` has the formulas) through ``_build/fg_torch.so``, the compiled
binding: at a few microseconds a call, doing that from Python would take most of
the time.  There is no fallback: if the binding has not been built, loading it
raises.  `stream` is a torch stream or a raw handle; None is the current one.
On another stream than the current one the caller orders only what it passes
and takes: that stream waits for the inputs, and whoever uses the outputs for
that stream.  Outputs and workspaces come from that stream's memory, and no
tensor's memory is reused before both are done with it.
"""
import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

import mx_gemm_gb300 as _fg
from mx_gemm_gb300 import build

BINDING_PATH = os.path.join(_fg.HERE, "_build", "fg_torch.so")
FG_TYPE_F32, FG_TYPE_BF16 = 0, 1
FG_ACT_NONE, FG_ACT_SWIGLU = 0, 1
FG_FLAG_RENORMALIZE = 0x1
_ACTS = {"none": FG_ACT_NONE, "swiglu": FG_ACT_SWIGLU}
_binding = None


def binding():
    """Load fg_torch.so (raises if it was not built, or for another torch)."""
    global _binding
    if _binding is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError("fg_torch.so is not built (%s); run mx_gemm_gb300.build.build()" % BINDING_PATH)
        if build.made_for() != build.running():  # it would be read with the wrong layouts of torch's classes
            raise RuntimeError("fg_torch.so was built for %s, this is %s; run mx_gemm_gb300.build.build()"
                               % ((build.made_for() or "another torch").strip(), build.running().strip()))
        _fg.lib()
        spec = importlib.util.spec_from_file_location("fg_torch", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_error(_fg.FgError)
        _binding = module
    return _binding


def binding_if_built():
    """The binding, or None where it has not been built, or for another torch."""
    if _binding is None and not (os.path.exists(BINDING_PATH) and build.made_for() == build.running()):
        return None
    return binding()


def _handle(stream):
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


class Routing(NamedTuple):
    """What moe_route returns (see fg_moe_route in include/fg.h)."""
    weights: torch.Tensor   # fp32 [T][top_k]
    experts: torch.Tensor   # int32 [T][top_k]
    offsets: torch.Tensor   # int32 [E + 1]
    rows: torch.Tensor      # int32 [T * top_k]: token of each slot
    slots: torch.Tensor     # int32 [T][top_k]: slot of each choice


def quantize(mode, x, act="none", stream=None):
    """(codes, scales) of the A operand of `mode` from x [M][K] (fp32 or bf16),
    or with act="swiglu" from rows (g, u) of 2K values.

    Codes are float8_e4m3fn [M][K] (uint8 [M][K/2], two e2m1 codes a byte, for
    mxfp4); scales float8_e8m0fnu [M][K/32] ([M][K/128] for mxfp8), or fp32
    [M][K/128] for fp8_block128.  The rows of x may be any distance apart.
    """
    return (_binding or binding()).quantize(_fg._mode(mode), _ACTS[act] if act in _ACTS else act, x, _handle(stream))


def rmsnorm_quantize(mode, x, weight, residual=None, eps=1e-6, normed=False, stream=None):
    """(codes, scales, h, y) of y = RMSnorm(h) * weight with h = x + residual.

    codes and scales as quantize() gives them (None for mode "bf16"); h, the new
    residual, is None where no residual is given; y is None unless `normed` is
    set or the mode is "bf16".  x, residual and weight are all fp32 or all bf16,
    and so are h and y.
    """
    return (_binding or binding()).rmsnorm_quantize(_fg._mode(mode), x, weight, residual, eps, normed, _handle(stream))


def moe_route_workspace_size(tokens, experts):
    b = ctypes.c_uint64()
    _fg._check(_fg.lib().fg_moe_route_workspace_size(tokens, experts, ctypes.byref(b)))
    return b.value


def moe_route(logits, top_k, renormalize=True, stream=None):
    """Routing of the tokens of logits [T][E] (fp32 or bf16) to top_k experts
    each: a Routing (weights, experts, offsets, rows, slots)."""
    return tuple.__new__(Routing, (_binding or binding()).moe_route(logits, top_k, renormalize, _handle(stream)))


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
    Rows of Y that no expert holds are left as they are.  A workspace is
    allocated here when one is needed and none is given.
    """
    return (_binding or binding()).grouped_gemm(A, pb.data, ctypes.addressof(pb.desc), offsets, a_scales, rows, Y, workspace,
                                                flags, _handle(stream))


def moe_combine(Y, slots, weights, residual=None, stream=None):
    """out[t] = residual[t] + sum_j weights[t][j] * Y[slots[t][j]] (bf16 [T][N])
    for the experts' rows Y [R][N]; a slot of -1 is no choice."""
    return (_binding or binding()).moe_combine(Y, slots, weights, residual, _handle(stream))
