"""Python binding of libtgemm_ffn.so: the operators of a model's feed-forward
layers around the dense products (include/tgemm_ffn.h states each).

As in the package itself, only arguments are marshalled: types, devices, shapes
and strides are checked, outputs and workspaces allocated when none are given,
and the C entry point of the same name is called on the tensors' device and on
that device's current stream unless a stream is given (what is allocated then
belongs to that stream).  That part is compiled (_ffn_binding, from
csrc/tgemm_ffn_binding.cpp): for a few tokens it would cost more than the
kernels.  There is no fallback: without the built libraries the first call
fails.

Matrices may have any row stride (last dimension contiguous) that is a multiple
of 8 elements.  Gradients are functions of their own, not autograd nodes.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import PKG_DIR, TgemmError, _torch

LIB_PATH = os.path.join(PKG_DIR, "libtgemm_ffn.so")
BINDING_PATH = os.path.join(PKG_DIR, "_ffn_binding.so")

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5, "geglu": 6}
SCORES = {"softmax": 0, "sigmoid": 1}

# The argument structs of include/tgemm_ffn.h, field by field in order: all
# are 8 bytes ("scale" and "eps" doubles, the rest integers or pointers).
_FIELDS = {
    "gemm_epilogue": "dtype trans_a trans_b M N K A lda B ldb bias residual ldr preact ldp C ldc act workspace "
                     "workspace_bytes",
    "gemm_epilogue_backward": "dtype M N dout ldd preact ldp act dz ldz dbias groups offsets workspace "
                              "workspace_bytes",
    "gemm_grouped": "dtype trans_b R N K groups offsets rows src_rows A lda B ldb stride_b bias preact ldp C ldc act",
    "gemm_grouped_tn": "dtype R P Q groups offsets X ldx Y ldy out",
    "route_topk": "dtype T E logits ld bias k score groups groups_used renormalize scale weights ids",
    "route_topk_backward": "dtype T E logits ld ids dweights k score renormalize scale dlogits ldo",
    "route_plan": "T k E ids offsets rows slots workspace workspace_bytes",
    "expert_gather": "R D src_rows x ldx rows out ldo",
    "expert_combine": "dtype T D R k h ldh slots weights residual ldr out ldo",
    "expert_combine_backward": "dtype T D R k dout ldd h ldh slots weights dh ldg dweights",
    "layer_norm": "dtype wdtype M N x ldx weight bias eps y ldy mean rstd",
    "layer_norm_backward": "dtype wdtype M N dy ldd x ldx weight mean rstd residual ldr dx ldo dweight dbias workspace "
                           "workspace_bytes",
    "quantize_mxfp4": "dtype M N x ldx q ldq scales qt ldqt scalest",
    "dequantize_mxfp4": "dtype M N q ldq scales out ldo",
    "gemm_mxfp4_epilogue": "dtype M N K A lda scale_A B ldb scale_B bias residual ldr preact ldp C ldc act workspace "
                           "workspace_bytes",
    "gemm_mxfp4_grouped": "dtype R N K groups offsets rows src_rows A lda scale_A B ldb stride_b scale_B stride_sb bias "
                          "preact ldp C ldc act",
}
_PACK = {n: struct.Struct("@" + "".join("d" if f in ("scale", "eps") else "q" for f in s.split())).pack
         for n, s in _FIELDS.items()}

_lib = None
_binding = None


def lib() -> ctypes.CDLL:
    """The loaded libtgemm_ffn.so with argument types set (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m dense_tiled_gemm_bf16_amd.build` "
            "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    i64 = ctypes.c_int64
    for name in _FIELDS:
        f = getattr(L, name)
        f.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        f.restype = ctypes.c_int
    L.tgemm_ffn_last_error.restype = ctypes.c_char_p
    L.tgemm_ffn_set_tile.argtypes = [ctypes.c_int, ctypes.c_int]
    L.tgemm_ffn_set_tile.restype = ctypes.c_int
    L.tgemm_epilogue_workspace_bytes.argtypes = [i64] * 5
    L.tgemm_epilogue_workspace_bytes.restype = ctypes.c_uint64
    for f in (L.tgemm_epilogue_backward_workspace_bytes, L.tgemm_route_plan_workspace_bytes):
        f.argtypes = [i64, i64, i64]
        f.restype = ctypes.c_uint64
    L.tgemm_mxfp4_workspace_bytes.argtypes = [i64, i64, i64]
    L.tgemm_layer_norm_backward_workspace_bytes.argtypes = [i64, i64]
    for f in (L.tgemm_mxfp4_workspace_bytes, L.tgemm_layer_norm_backward_workspace_bytes):
        f.restype = ctypes.c_uint64
    _lib = L
    return L


def binding():
    """The compiled module (raises if not built)."""
    global _binding
    if _binding is None:
        import importlib.machinery
        import importlib.util

        lib()
        _torch()      # its libraries are what the module links to
        if not os.path.exists(BINDING_PATH):
            raise ImportError(f"{BINDING_PATH} is not built; run `python -m dense_tiled_gemm_bf16_amd.build` first")
        loader = importlib.machinery.ExtensionFileLoader("_ffn_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ffn_binding", loader))
        loader.exec_module(module)
        module.set_error(TgemmError)
        _binding = module
    return _binding


def args(name: str, **fields) -> bytes:
    """The argument struct of a C entry point (fields not given are 0)."""
    order = _FIELDS[name].split()
    unknown = set(fields) - set(order)
    if unknown:
        raise TypeError(f"{name} has no field {sorted(unknown)}")
    return _PACK[name](*(fields.get(f) or 0 for f in order))


def last_error() -> str:
    return lib().tgemm_ffn_last_error().decode()


def set_tile(tile_m: int = 0, tile_n: int = 0) -> None:
    """Force the output tile of this thread's later products here; (0, 0)
    restores the library's own choice (tgemm_ffn_set_tile)."""
    rc = lib().tgemm_ffn_set_tile(tile_m, tile_n)
    if rc != 0:
        raise TgemmError(rc, last_error())


def _call(name, first, stream, *values):
    """The compiled function, with the given stream current."""
    f = getattr(_binding or binding(), name)
    if stream is None:
        return f(*values)
    torch = _torch()
    if isinstance(first, torch.Tensor) and stream.device != first.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
    with torch.cuda.stream(stream):
        return f(*values)


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return code


def _score(score):
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return code


def gemm_epilogue(a, b, bias=None, act="none", residual=None, preact=None, out=None, workspace=None, stream=None):
    """act(a @ b + bias) + residual for 2-D bfloat16 or float16 CUDA tensors.

    a (M,K) and b (K,N) as in gemm(): row-major or the transpose of a row-major
    array.  bias (N,), residual and out in the input type.  act: "none",
    "relu", "gelu" (erf), "gelu_tanh", "silu", or gated: "swiglu", "geglu"
    take b = [gate | up] and give (M, N/2) (a row-major then).  preact (M,N), if
    given, receives a @ b + bias for epilogue_backward.  residual may be out.
    workspace: for a K split, tgemm_epilogue_workspace_bytes bytes (with less
    there is none); allocated when None.
    """
    return _call("gemm_epilogue", a, stream, a, b, bias, _act(act), residual, preact, out,
                 workspace)


def epilogue_backward(dout, preact, act, offsets=None, want_dbias=True, dz=None, dbias=None, workspace=None,
                      stream=None):
    """Backward pass of the epilogue: (dz, dbias).

    dout: the gradient of act(z); preact: z as gemm_epilogue kept it (None for
    act "none", whose dz is dout itself unless a dz is given).  dbias is the
    column sums (N,), or (groups, N) over the row groups of `offsets`
    (groups + 1,) int32; None if not wanted.  Rows in no group are not
    written.  workspace: a uint8 tensor of
    tgemm_epilogue_backward_workspace_bytes; allocated when None.
    """
    return _call("epilogue_backward", dout, stream, dout, preact, _act(act), offsets, want_dbias, dz, dbias,
                 workspace)


def gemm_grouped(a, b, offsets, rows=None, bias=None, act="none", preact=None, out=None, stream=None):
    """The experts' products: out[r] = act(a[rows[r]] @ b[e] + bias[e]) for each
    row r of group e, the rows offsets[e] .. offsets[e + 1] - 1.

    a (S,K) row-major; b (E,K,N), each b[e] row-major or transposed (weights
    kept (E,N,K) go in as ``w.transpose(1, 2)``); offsets (E + 1,) and rows (R,)
    int32 on the device (rows None: R = S, row r itself; an index outside a
    reads zeros).  bias (E,N); act, preact (R,N) and out (R,N or N/2) as in
    gemm_epilogue.  Rows in no group are not written.
    """
    return _call("gemm_grouped", a, stream, a, b, offsets, rows, bias, _act(act), preact, out)


def gemm_grouped_tn(x, y, offsets, out=None, stream=None):
    """out[e] = x_e.T @ y_e over the rows of group e: x (R,P), y (R,Q) ->
    (E,P,Q), zeros for an empty group (the experts' weight gradients)."""
    return _call("gemm_grouped_tn", x, stream, x, y, offsets, out)


def route_topk(logits, k, score="softmax", bias=None, groups=1, groups_used=1, renormalize=True, scale=1.0,
               weights=None, ids=None, stream=None):
    """The k experts of each token: (weights (T,k) float32, ids (T,k) int32).

    logits (T,E) float32, bfloat16 or float16, rows of any stride.  Scores are
    the softmax or sigmoid of the logits; chosen are the largest score + bias
    (bias (E,) float32), with groups > 1 only from the groups_used groups whose
    two largest are highest; ties go to the lowest expert.  weights: the chosen
    scores, divided by their sum if renormalize (sigmoid: their sum + 1e-20),
    times scale.  Logits of -inf or NaN are never chosen; missing choices have
    id -1 and weight 0.
    """
    return _call("route_topk", logits, stream, logits, k, _score(score), bias, groups, groups_used, renormalize, scale,
                 weights, ids)


def route_topk_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, dlogits=None,
                        stream=None):
    """The gradient of route_topk's weights with respect to the logits, from
    dweights (T,k) float32, the logits and the ids it gave (distinct in a
    row): dlogits (T,E) in the logits' type, and may be logits."""
    return _call("route_topk_backward", logits, stream, dweights, logits, ids, _score(score), renormalize, scale, dlogits)


def route_plan(ids, experts, offsets=None, rows=None, slots=None, workspace=None, stream=None):
    """The choices (T,k) int32 sorted by expert: (offsets (experts + 1,), rows
    (T k,), slots (T,k)), all int32: the row groups, the token of each row (-1
    behind the last) and the row of each choice (-1 for an id outside the
    experts)."""
    return _call("route_plan", ids, stream, ids, experts, offsets, rows, slots, workspace)


def expert_gather(x, rows, out=None, stream=None):
    """out[r] = x[rows[r]]: the experts' rows side by side (x (T,D) of a 16-bit
    type, rows (R,) int32).  A row whose index is outside x is not written."""
    return _call("expert_gather", x, stream, x, rows, out)


def expert_combine(h, slots, weights=None, residual=None, out=None, stream=None):
    """out[t] = sum over j of weights[t,j] h[slots[t,j]] + residual[t]: h (R,D)
    of a 16-bit type, slots (T,k) int32 (outside 0 .. R - 1: nothing), weights
    (T,k) float32 or None for ones.  Without weights it is the gradient of
    expert_gather.  residual may be out."""
    return _call("expert_combine", h, stream, h, slots, weights, residual, out)


def expert_combine_backward(dout, h, slots, weights, dh=None, dweights=None, stream=None):
    """Gradients of expert_combine: (dh (R,D), dweights (T,k) float32).  Rows
    of dh that no slot names are not written; slots are to be distinct, as a
    plan's are (a row that several name holds no sum of theirs)."""
    return _call("expert_combine_backward", dout, stream, dout, h, slots, weights, dh, dweights)


def layer_norm(x, weight=None, bias=None, eps=1e-5, mean=None, rstd=None, out=None, stream=None):
    """(x - mean) / sqrt(var + eps) * weight + bias over the rows of x (M,N),
    bfloat16, float16 or float32; var is the mean squared difference.

    weight and bias (N,) in x's type or both float32 (None: ones, zeros).  mean
    and rstd (M,) float32, if given, receive each row's mean and 1 / sqrt(var +
    eps), for layer_norm_backward.  out may be x.
    """
    return _call("layer_norm", x, stream, x, weight, bias, eps, mean, rstd, out)


def layer_norm_backward(dout, x, weight, mean, rstd, residual=None, want_dweight=True, dx=None, dweight=None, dbias=None,
                        workspace=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias).

    mean, rstd: as layer_norm left them; weight as there (None: ones).
    residual (M,N), if given, is added to dx (a gradient that reaches x another
    way).  dweight and dbias (N,) have the weight's type (x's without one); None
    if not wanted.  dx may be dout, x or residual.  workspace: a uint8
    tensor of tgemm_layer_norm_backward_workspace_bytes; allocated when None.
    """
    return _call("layer_norm_backward", x, stream, dout, x, weight, mean, rstd, residual, want_dweight, dx, dweight, dbias,
                 workspace)


def quantize_mxfp4(x, rows=True, columns=False, q=None, scales=None, qt=None, scalest=None, stream=None):
    """MXFP4 operands of x (M,N), bfloat16, float16 or float32.

    rows: (q (M,N/2), scales (M,N/32)), uint8, as gemm_mxfp4_nt and
    gemm_mxfp4_epilogue take them, one scale per 32 values of a row.  columns:
    (qt (N,P/2), scalest (N,P/32)), the same of x.t(), zeros behind its M
    values up to P, M rounded up to 32: what the products of a backward pass
    take; the rows of a qt made here are a multiple of 128 bytes apart.  Both, in
    one read of x: (q, scales, qt, scalest).  A block with an infinity or a NaN
    becomes NaN.
    """
    return _call("quantize_mxfp4", x, stream, x, rows, columns, q, scales, qt, scalest)


_dtypes = {}  # (made once: in every call it took as long as an allocation, 0.6 us)


def _dtype(dtype):
    if not _dtypes:
        torch = _torch()
        _dtypes.update({None: -1, torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _dtypes.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be torch.bfloat16, torch.float16 or torch.float32, got {dtype!r}")
    return code


def dequantize_mxfp4(q, scales, dtype=None, out=None, stream=None):
    """The values of MXFP4 rows q (M,N/2), scales (M,N/32): (M,N) in dtype
    (torch.bfloat16 when None; out's if one is given), which holds each below
    2^128 exactly unless it is float16.  Values past the type's largest are
    infinite: elements 4 and 6 at scale byte 253, 2 to 6 at 254; a finite number
    from 1.75 2^127 on is quantised to such a one."""
    return _call("dequantize_mxfp4", q, stream, q, scales, _dtype(dtype), out)


def gemm_mxfp4_epilogue(a, b, scale_a, scale_b, bias=None, act="none", residual=None, preact=None, out=None, dtype=None,
                        workspace=None, stream=None):
    """act(a @ b.T + bias) + residual on MXFP4 operands: gemm_epilogue's epilogue on
    gemm_mxfp4_nt's product, for any M from 1.

    a (M,K/2), b (N,K/2): packed E2M1 bytes (uint8), rows of any stride that is a
    multiple of 16; scale_a (M,K/32), scale_b (N,K/32): e8m0 bytes, contiguous.
    bias, act, residual, preact as in gemm_epilogue, in dtype (bfloat16 or
    float16; when None that of out, bias, residual or preact, else bfloat16).
    workspace: for a K split, tgemm_mxfp4_workspace_bytes bytes (with less
    there is none); allocated when None.
    """
    return _call("gemm_mxfp4_epilogue", a, stream, a, b, scale_a, scale_b, bias, _act(act), residual, preact, out,
                 _dtype(dtype), workspace)


def gemm_mxfp4_grouped(a, b, scale_a, scale_b, offsets, rows=None, bias=None, act="none", preact=None, out=None, dtype=None,
                       stream=None):
    """gemm_grouped on MXFP4 operands: out[r] = act(a[rows[r]] @ b[e].T + bias[e])
    for each row r of group e.

    a (S,K/2), scale_a (S,K/32); b (E,N,K/2), scale_b (E,N,K/32), each
    scale_b[e] contiguous; offsets, rows, bias, act, preact, out as in
    gemm_grouped, dtype as in gemm_mxfp4_epilogue.  Rows in no group are not
    written.
    """
    return _call("gemm_mxfp4_grouped", a, stream, a, b, scale_a, scale_b, offsets, rows, bias, _act(act), preact, out,
                 _dtype(dtype))
