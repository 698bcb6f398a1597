"""Python binding of libfp8moe: expert routing with its gradients, and the
W8A8 layers in 8-bit integers (C ABI: include/fp8moe.h).

As in the package itself, argument marshalling only: checks, outputs and the
sort's workspace allocated with torch, the current torch stream of the
tensors' device.  The calls go through a small native module
(csrc_moe/binding.cpp), since those of a decode step are bound by the host.
There is no fallback: if libfp8moe.so or the module is missing the functions
raise on first use.  Nothing here records a gradient: the backward passes are
calls of their own, and tensors that require a gradient are refused except
under torch.no_grad() or in a torch.autograd.Function.  Outputs given by the
caller share no memory with each other or with inputs; 2-D tensors may have any
row stride unless stated.  New outputs of one call may be parts of one small
allocation (up to 1 MB): copy one before it is resized in place.  No row is
named twice in token_rows.
"""
import ctypes
import os
from typing import NamedTuple

import torch

from . import Fp8Error

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8moe.so")

_moe_lib = None


def moe_lib():
    """The loaded libfp8moe.so (raises if it has not been built)."""
    global _moe_lib
    if _moe_lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m fp8_block_scaled_02_amd.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.fp8b_moe_abi_version.restype = ci
        L.fp8b_moe_abi_version.argtypes = []
        L.moe_sort_workspace.restype = i64
        L.moe_sort_workspace.argtypes = [i64, i64, i64]
        for name, args in (
                ("moe_route", [vp, ci, i64, i64, i64, i64, ci] + [vp] * 7),
                ("moe_sort", [vp, i64, i64, i64] + [vp] * 5),
                ("moe_route_backward", [vp, vp, ci, i64, vp, vp, i64, i64, i64, ci, vp, i64, vp]),
                ("moe_gather", [vp, ci, i64, i64, i64, vp, i64, i64, vp, i64, vp]),
                ("moe_combine", [vp, ci, i64, i64, i64, vp, vp, i64, i64, vp, ci, i64, vp]),
                ("moe_combine_backward", [vp, ci, i64, vp, ci, i64, i64, i64, vp, vp, i64, i64, vp, i64, vp, vp]),
                ("int8_quant", [vp, ci, i64, i64, i64, vp, i64, vp, vp]),
                ("int8_weight_pack", [vp, i64, i64, i64, i64, i64, vp, vp]),
                ("int8_gemm", [vp, i64, vp, vp, vp, vp, i64, i64, i64, vp, i64, ci, vp]),
                ("int8_grouped_gemm", [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, i64, i64, vp, i64, ci, vp])):
            getattr(L, name).restype = ci
            getattr(L, name).argtypes = args
        _moe_lib = L
    return _moe_lib


_native = None
_current_device = _raw_stream = None    # torch's device calls, looked up with the native module


def _load():
    """The native module of the calls below (raises if it has not been built)."""
    global _native, _current_device, _raw_stream
    if _native is None:
        moe_lib()
        try:
            from . import _moe_binding
        except ImportError as e:
            raise ImportError(f"{e}: build it with `python -m fp8_block_scaled_02_amd.build` "
                              "(there is no Python fallback)") from e
        _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _native = _moe_binding
    return _native


_C_NAMES = {"route": "moe_route", "sort": "moe_sort", "route_backward": "moe_route_backward", "gather": "moe_gather",
            "combine": "moe_combine", "combine_backward": "moe_combine_backward", "quant": "int8_quant",
            "pack": "int8_weight_pack", "gemm": "int8_gemm", "grouped": "int8_grouped_gemm", "linear": "int8_linear",
            "forward": "int8_moe_forward"}


def _call(fn, first, *args):
    """One native call on the current stream of the GPU of tensor `first`,
    which is made current for it: a default stream is NULL, which means the
    current device's.  (A host tensor is refused by the call.)"""
    f = getattr(_native or _load(), fn)
    dev = first.get_device()
    if dev < 0:
        out = f(0, first, *args)
    elif dev == _current_device():
        out = f(_raw_stream(dev), first, *args)
    else:
        with torch.cuda.device(dev):
            out = f(_raw_stream(dev), first, *args)
    if out.__class__ is int:
        raise Fp8Error(_C_NAMES[fn], out)
    return out


def _fp32(dtype, name="out_dtype"):
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return dtype is torch.float32


class Routing(NamedTuple):
    """What moe_route makes for T tokens, k slots each, and E experts; R = T * k
    rows in the order of (expert, token, slot).  -1 stands for none."""
    gates: torch.Tensor            # float32 [T, k]  weights, 0 for an empty slot
    experts: torch.Tensor          # int32 [T, k]    each slot's expert
    expert_offsets: torch.Tensor   # int32 [E + 1]   rows of expert e: from [e] to [e + 1]
    row_index: torch.Tensor        # int32 [R]       each row's token
    token_rows: torch.Tensor       # int32 [T, k]    each slot's row


def moe_route(logits, k: int, renormalize: bool = True) -> Routing:
    """Each token's k experts of the largest logits (fp32 or bf16 [T, E], the
    lower id first among equal ones) and their softmax weights, over the chosen
    ones (renormalize) or over all E, with the plan that sorts the slots by
    expert.  A logit of -inf is never chosen: a padding token's are all -inf."""
    return Routing(*_call("route", logits, k, renormalize))


def moe_sort(experts, num_experts: int):
    """The plan alone, for experts int32 [T, k] chosen elsewhere (ids outside
    0 .. num_experts - 1: no row): (expert_offsets, row_index, token_rows)."""
    return _call("sort", experts, num_experts)


def moe_route_backward(dgates, logits, gates, experts, renormalize: bool = True, out=None):
    """The logits' gradient [T, E], in their type, from that of moe_route's
    gates (dgates float32 [T, k])."""
    return _call("route_backward", dgates, logits, gates, experts, renormalize, out)


def moe_gather(x, token_rows, rows=None, out=None):
    """Token rows to their experts: out[token_rows[t, j]] = x[t], x bf16 or
    fp32 [T, N].  rows: how many there are (T * k, or those of out).  Rows that
    no slot names are left as they were."""
    return _call("gather", x, token_rows, rows, out)


def moe_gather_backward(drows, token_rows, out=None):
    """The gradient of moe_gather: the sum of each token's rows of drows
    [R, N], in fp32, rounded once to their type."""
    return _call("combine", drows, token_rows, None, None, out)


def moe_combine(y, token_rows, gates, out_dtype=None, out=None):
    """Rows back to their tokens, weighted: out[t] = sum_j gates[t, j] *
    y[token_rows[t, j]] over the slots that have a row, in fp32; y bf16 or
    fp32 [R, N], gates float32 [T, k].  out_dtype defaults to y's."""
    if gates is None:
        raise ValueError("gates must be a tensor")
    return _call("combine", y, token_rows, gates, None if out_dtype is None else _fp32(out_dtype), out)


def moe_combine_backward(dout, y, token_rows, gates, dy=None, dgates=None):
    """The gradients of moe_combine: (dy [R, N] in y's type, dgates float32
    [T, k]).  Rows of dy that no slot names are left as they were (of a new dy:
    undefined)."""
    return _call("combine_backward", dout, y, token_rows, gates, dy, dgates)


def int8_quant(x, codes=None, scales=None):
    """One scale per row: x bf16 or fp32 [M, K] -> (codes int8 [M, K], scales
    float32 [M]), codes the nearest whole numbers to x / (amax / 127).  New
    codes have their rows whole 128-byte lines apart, as the products read
    them."""
    return _call("quant", x, codes, scales)


def int8_weight_pack(w, out=None):
    """Weight codes int8 [N, K] or [E, N, K] into the layout that the products
    read (1 KB chunks of 16 rows x 64 codes, K outermost), filled up with zeros
    to multiples of 16 rows and 128 columns."""
    return _call("pack", w, out)


def int8_gemm(a, a_scales, w_packed, w_scales, bias=None, out_dtype=torch.bfloat16, y=None):
    """y[M, N] = (a . w) * a_scales * w_scales (+ bias): codes a int8 [M, K] as
    int8_quant lays them out, w_packed from int8_weight_pack, scales float32
    [M] and [N], bias float32 [N].  The sums are exact."""
    return _call("gemm", a, a_scales, w_packed, w_scales, bias, _fp32(out_dtype), y)


def int8_grouped_gemm(a, a_scales, row_index, expert_offsets, w_packed, w_scales, out_dtype=torch.bfloat16, y=None):
    """int8_gemm per expert with the gather inside: row r of expert e is
    a[row_index[r]] (row_index None: row r itself, a in expert order) times
    that expert's weights, w_packed from int8_weight_pack of [E, N, K].  Rows
    of y from expert_offsets[E] on are left as they were."""
    return _call("grouped", a, a_scales, row_index, expert_offsets, w_packed, w_scales, _fp32(out_dtype), y)


def int8_linear(x, w_packed, w_scales, bias=None, out_dtype=torch.bfloat16):
    """W8A8 linear layer in 8-bit integers: int8_quant(x), then int8_gemm."""
    return _call("linear", x, w_packed, w_scales, bias, _fp32(out_dtype))


def int8_moe_forward(x, logits, k: int, w_packed, w_scales, renormalize: bool = True, out_dtype=None, rows_dtype=None):
    """One expert projection: moe_route of the logits, int8_quant of the
    tokens, int8_grouped_gemm, moe_combine.  Returns (out [T, N], the Routing).
    With neither type given the experts' rows are held in fp32, and only the
    output is rounded, once, to bf16.  out_dtype is the type of both, so that
    bf16 rows are rounded before their sum and take half the bytes; rows_dtype
    gives the rows' own."""
    if rows_dtype is None:
        rows_dtype = torch.float32 if out_dtype is None else out_dtype
    out = _call("forward", x, logits, k, w_packed, w_scales, renormalize, _fp32(rows_dtype, "rows_dtype"),
                out_dtype is not None and _fp32(out_dtype))
    return out[0], Routing(*out[1:])
