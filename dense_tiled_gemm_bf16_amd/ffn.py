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
# are 8 bytes ("scale" a double, the rest integers or pointers).
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
}
_PACK = {n: struct.Struct("@" + "".join("d" if f == "scale" else "q" for f in s.split())).pack
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
