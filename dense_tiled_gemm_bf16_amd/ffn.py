"""Python binding of libtgemm_ffn.so: the operators of a model's feed-forward
layers around the dense products (include/tgemm_ffn.h states each).

As in the package itself, only arguments are marshalled here: types, devices,
shapes and strides are checked, outputs and workspaces allocated when none are
given, and the C entry point of the same name is called on the tensors' device
and on that device's current stream unless a stream is given (what is
allocated here then belongs to that stream).  There is no fallback: without
the built library the first call fails.

Matrices may have any row stride (last dimension contiguous) that is a multiple
of 8 elements.  Gradients are functions of their own, not autograd nodes.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import PKG_DIR, TgemmError, _layout, _torch

LIB_PATH = os.path.join(PKG_DIR, "libtgemm_ffn.so")

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5, "geglu": 6}
GATED = ("swiglu", "geglu")
SCORES = {"softmax": 0, "sigmoid": 1}

# The argument structs of include/tgemm_ffn.h, field by field in order: all
# are 8 bytes ("scale" a double, the rest integers or pointers).
_FIELDS = {
    "gemm_epilogue": "dtype trans_a trans_b M N K A lda B ldb bias residual ldr preact ldp C ldc act",
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
_fn = {}


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
        _fn[name] = f
    L.tgemm_ffn_last_error.restype = ctypes.c_char_p
    L.tgemm_ffn_set_tile.argtypes = [ctypes.c_int, ctypes.c_int]
    L.tgemm_ffn_set_tile.restype = ctypes.c_int
    for f in (L.tgemm_epilogue_backward_workspace_bytes, L.tgemm_route_plan_workspace_bytes):
        f.argtypes = [i64, i64, i64]
        f.restype = ctypes.c_uint64
    _lib = L
    return L


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


class _On:
    """The device of a call's tensors and the stream it goes to."""

    __slots__ = ("torch", "device", "index", "stream")

    def __init__(self, first, stream):
        torch = _torch()
        if not isinstance(first, torch.Tensor):
            raise TypeError("operands must be torch tensors")
        if not first.is_cuda:
            raise ValueError("operands must be on a GPU")
        if _lib is None:
            lib()
        self.torch = torch
        self.device = first.device
        self.index = self.device.index
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {self.device}")
        self.stream = stream

    def new(self, shape, dtype):
        if self.stream is None:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        with self.torch.cuda.stream(self.stream):
            return self.torch.empty(shape, dtype=dtype, device=self.device)

    def same(self, t, name):
        if not isinstance(t, self.torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, not on {self.device} with the other operands")

    def mat(self, t, name, dtype, rows, cols):
        """Row stride of a (rows, cols) matrix with contiguous rows."""
        self.same(t, name)
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != (rows, cols):
            raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
        s0, s1 = t.stride()
        if (s1 != 1 and cols > 1) or (rows > 1 and s0 < cols):
            raise ValueError(f"{name} must be row-major (strides {(s0, s1)})")
        return max(s0, cols)

    def packed(self, t, name, dtype, shape):
        self.same(t, name)
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def call(self, name, *values):
        torch = self.torch
        packed = _PACK[name](*values)
        if torch.cuda.current_device() == self.index:
            rc = _fn[name](packed, self._stream())
        else:
            with torch.cuda.device(self.index):
                rc = _fn[name](packed, self._stream())
        if rc != 0:
            raise TgemmError(rc, last_error())

    def _stream(self):
        if self.stream is not None:
            return self.stream.cuda_stream
        return self.torch._C._cuda_getCurrentRawStream(self.index)


def _dtype16(t, name):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def _dtype_logits(t):
    return 2 if t.dtype == _torch().float32 else _dtype16(t, "logits")


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


def _halved(n, act):
    if act not in GATED:
        return n
    if n % 2:
        raise ValueError(f"a gated activation takes an even number of columns, got {n}")
    return n // 2


def gemm_epilogue(a, b, bias=None, act="none", residual=None, preact=None, out=None, stream=None):
    """act(a @ b + bias) + residual for 2-D bfloat16 or float16 CUDA tensors.

    a (M,K) and b (K,N) as in gemm(): row-major or the transpose of a row-major
    array.  bias (N,), residual and out in the input type.  act: "none",
    "relu", "gelu" (erf), "gelu_tanh", "silu", or gated: "swiglu", "geglu"
    take b = [gate | up] and give (M, N/2) (a row-major then).  preact (M,N), if
    given, receives a @ b + bias for epilogue_backward.  residual may be out.
    """
    on = _On(a, stream)
    if a.dim() != 2 or not isinstance(b, on.torch.Tensor) or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError("a and b must be matrices that multiply")
    dt = _dtype16(a, "a")
    if b.dtype != a.dtype:
        raise TypeError("a and b must both be bfloat16 or both float16")
    on.same(b, "b")
    M, K = a.shape
    N = b.shape[1]
    code = _act(act)
    F = _halved(N, act)
    ta, lda = _layout(a, "a")
    tb, ldb = _layout(b, "b")
    dtype = a.dtype
    pb = on.packed(bias, "bias", dtype, (N,)) if bias is not None else 0
    pr = ldr = pp = ldp = 0
    if residual is not None:
        ldr, pr = on.mat(residual, "residual", dtype, M, F), residual.data_ptr()
    if preact is not None:
        ldp, pp = on.mat(preact, "preact", dtype, M, N), preact.data_ptr()
    if out is None:
        out, ldc = on.new((M, F), dtype), F
    else:
        ldc = on.mat(out, "out", dtype, M, F)
    on.call("gemm_epilogue", dt, ta, tb, M, N, K, a.data_ptr(), lda, b.data_ptr(), ldb, pb, pr, ldr, pp, ldp,
            out.data_ptr(), ldc, code)
    return out


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
    on = _On(dout, stream)
    dt = _dtype16(dout, "dout")
    if dout.dim() != 2:
        raise ValueError("dout must be a matrix")
    dtype = dout.dtype
    M, F = dout.shape
    code = _act(act)
    N = 2 * F if act in GATED else F
    ldd = on.mat(dout, "dout", dtype, M, F)
    pp = ldp = pz = ldz = po = pb = pw = nw = groups = 0
    if code != 0:
        if preact is None:
            raise ValueError(f"act {act!r} needs preact")
        ldp, pp = on.mat(preact, "preact", dtype, M, N), preact.data_ptr()
    if dz is not None:
        ldz, pz = on.mat(dz, "dz", dtype, M, N), dz.data_ptr()
    elif code != 0:
        dz = on.new((M, N), dtype)
        ldz, pz = N, dz.data_ptr()
    if offsets is not None:
        groups = offsets.numel() - 1
        if groups < 1:
            raise ValueError("offsets must hold groups + 1 entries")
        po = on.packed(offsets, "offsets", on.torch.int32, (groups + 1,))
    if want_dbias:
        shape = (groups, N) if groups else (N,)
        if dbias is None:
            dbias = on.new(shape, dtype)
        pb = on.packed(dbias, "dbias", dtype, shape)
        need = _lib.tgemm_epilogue_backward_workspace_bytes(M, N, groups)
        if workspace is None:
            workspace = on.new((max(need, 16),), on.torch.uint8)
        on.same(workspace, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        pw, nw = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    on.call("gemm_epilogue_backward", dt, M, N, dout.data_ptr(), ldd, pp, ldp, code, pz, ldz, pb, groups, po, pw, nw)
    return (dout if dz is None else dz), (dbias if want_dbias else None)


def _weights3(on, b, name, dtype):
    """(transposed, leading dimension, stride) of (E, K, N) matrices, each
    row-major or the transpose of a row-major one."""
    on.same(b, name)
    if b.dim() != 3:
        raise ValueError(f"{name} must be (groups, K, N)")
    if b.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {b.dtype}")
    _, r, c = b.shape
    se, s0, s1 = b.stride()
    if s1 == 1 and (s0 >= c or r == 1):
        return 0, max(s0, c), se
    if s0 == 1 and (s1 >= r or c == 1):
        return 1, max(s1, r), se
    raise ValueError(f"{name} must hold row-major or transposed row-major matrices (strides {b.stride()})")


def gemm_grouped(a, b, offsets, rows=None, bias=None, act="none", preact=None, out=None, stream=None):
    """The experts' products: out[r] = act(a[rows[r]] @ b[e] + bias[e]) for each
    row r of group e, the rows offsets[e] .. offsets[e + 1] - 1.

    a (S,K) row-major; b (E,K,N), each b[e] row-major or transposed (weights
    kept (E,N,K) go in as ``w.transpose(1, 2)``); offsets (E + 1,) and rows (R,)
    int32 on the device (rows None: R = S, row r itself; an index outside a
    reads zeros).  bias (E,N); act, preact (R,N) and out (R,N or N/2) as in
    gemm_epilogue.  Rows in no group are not written.
    """
    on = _On(a, stream)
    dt = _dtype16(a, "a")
    if a.dim() != 2:
        raise ValueError("a must be a matrix")
    dtype = a.dtype
    S, K = a.shape
    lda = on.mat(a, "a", dtype, S, K)
    tb, ldb, stride_b = _weights3(on, b, "b", dtype)
    E, Kb, N = b.shape
    if Kb != K:
        raise ValueError(f"a has {K} columns, b {Kb} rows")
    code = _act(act)
    F = _halved(N, act)
    int32 = on.torch.int32
    po = on.packed(offsets, "offsets", int32, (E + 1,))
    R, pi = S, 0
    if rows is not None:
        R = rows.numel()
        pi = on.packed(rows, "rows", int32, (R,))
    pb = on.packed(bias, "bias", dtype, (E, N)) if bias is not None else 0
    pp = ldp = 0
    if preact is not None:
        ldp, pp = on.mat(preact, "preact", dtype, R, N), preact.data_ptr()
    if out is None:
        out, ldc = on.new((R, F), dtype), F
    else:
        ldc = on.mat(out, "out", dtype, R, F)
    on.call("gemm_grouped", dt, tb, R, N, K, E, po, pi, S, a.data_ptr(), lda, b.data_ptr(), ldb, stride_b, pb, pp,
            ldp, out.data_ptr(), ldc, code)
    return out


def gemm_grouped_tn(x, y, offsets, out=None, stream=None):
    """out[e] = x_e.T @ y_e over the rows of group e: x (R,P), y (R,Q) ->
    (E,P,Q), zeros for an empty group (the experts' weight gradients)."""
    on = _On(x, stream)
    dt = _dtype16(x, "x")
    if x.dim() != 2 or not isinstance(y, on.torch.Tensor) or y.dim() != 2 or x.shape[0] != y.shape[0]:
        raise ValueError("x and y must be matrices of as many rows")
    dtype = x.dtype
    R, P = x.shape
    Q = y.shape[1]
    ldx = on.mat(x, "x", dtype, R, P)
    ldy = on.mat(y, "y", dtype, R, Q)
    E = offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must hold groups + 1 entries")
    po = on.packed(offsets, "offsets", on.torch.int32, (E + 1,))
    if out is None:
        out = on.new((E, P, Q), dtype)
    pc = on.packed(out, "out", dtype, (E, P, Q))
    on.call("gemm_grouped_tn", dt, R, P, Q, E, po, x.data_ptr(), ldx, y.data_ptr(), ldy, pc)
    return out


def route_topk(logits, k, score="softmax", bias=None, groups=1, groups_used=1, renormalize=True, scale=1.0,
               weights=None, ids=None, stream=None):
    """The k experts of each token: (weights (T,k) float32, ids (T,k) int32).

    logits (T,E) float32, bfloat16 or float16, rows of any stride.  Scores are
    the softmax or sigmoid of the logits; chosen are the largest score + bias
    (bias (E,) float32), with groups > 1 only from the groups_used groups whose
    two largest are highest; ties go to the lowest expert.  weights: the chosen
    scores, divided by their sum if renormalize, times scale.  Logits of -inf
    or NaN are never chosen; missing choices have id -1 and weight 0.
    """
    on = _On(logits, stream)
    dt = _dtype_logits(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix")
    T, E = logits.shape
    torch = on.torch
    ld = on.mat(logits, "logits", logits.dtype, T, E)
    pb = on.packed(bias, "bias", torch.float32, (E,)) if bias is not None else 0
    weights = on.new((T, k), torch.float32) if weights is None else weights
    ids = on.new((T, k), torch.int32) if ids is None else ids
    pw = on.packed(weights, "weights", torch.float32, (T, k))
    pi = on.packed(ids, "ids", torch.int32, (T, k))
    on.call("route_topk", dt, T, E, logits.data_ptr(), ld, pb, k, _score(score), groups, groups_used,
            int(renormalize), float(scale), pw, pi)
    return weights, ids


def route_topk_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, dlogits=None,
                        stream=None):
    """The gradient of route_topk's weights with respect to the logits, from
    dweights (T,k) float32, the logits and the ids it gave: dlogits (T,E) in
    the logits' type."""
    on = _On(logits, stream)
    dt = _dtype_logits(logits)
    if logits.dim() != 2 or not isinstance(ids, on.torch.Tensor) or ids.dim() != 2:
        raise ValueError("logits and ids must be matrices")
    T, E = logits.shape
    k = ids.shape[1]
    torch = on.torch
    ld = on.mat(logits, "logits", logits.dtype, T, E)
    pi = on.packed(ids, "ids", torch.int32, (T, k))
    pw = on.packed(dweights, "dweights", torch.float32, (T, k))
    dlogits = on.new((T, E), logits.dtype) if dlogits is None else dlogits
    ldo = on.mat(dlogits, "dlogits", logits.dtype, T, E)
    on.call("route_topk_backward", dt, T, E, logits.data_ptr(), ld, pi, pw, k, _score(score), int(renormalize),
            float(scale), dlogits.data_ptr(), ldo)
    return dlogits


def route_plan(ids, experts, offsets=None, rows=None, slots=None, workspace=None, stream=None):
    """The choices (T,k) int32 sorted by expert: (offsets (experts + 1,), rows
    (T k,), slots (T,k)), all int32: the row groups, the token of each row (-1
    behind the last) and the row of each choice (-1 for an id outside the
    experts)."""
    on = _On(ids, stream)
    int32 = on.torch.int32
    if ids.dim() != 2:
        raise ValueError("ids must be a matrix")
    T, k = ids.shape
    pi = on.packed(ids, "ids", int32, (T, k))
    offsets = on.new((experts + 1,), int32) if offsets is None else offsets
    rows = on.new((T * k,), int32) if rows is None else rows
    slots = on.new((T, k), int32) if slots is None else slots
    need = _lib.tgemm_route_plan_workspace_bytes(T, k, experts)
    pw = nw = 0
    if workspace is None and need:
        workspace = on.new((need,), on.torch.uint8)
    if workspace is not None:
        on.same(workspace, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        pw, nw = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    on.call("route_plan", T, k, experts, pi, on.packed(offsets, "offsets", int32, (experts + 1,)),
            on.packed(rows, "rows", int32, (T * k,)), on.packed(slots, "slots", int32, (T, k)), pw, nw)
    return offsets, rows, slots


def expert_gather(x, rows, out=None, stream=None):
    """out[r] = x[rows[r]]: the experts' rows side by side (x (T,D) of a 16-bit
    type, rows (R,) int32).  A row whose index is outside x is not written."""
    on = _On(x, stream)
    _dtype16(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    T, D = x.shape
    R = rows.numel()
    ldx = on.mat(x, "x", x.dtype, T, D)
    pi = on.packed(rows, "rows", on.torch.int32, (R,))
    out = on.new((R, D), x.dtype) if out is None else out
    ldo = on.mat(out, "out", x.dtype, R, D)
    on.call("expert_gather", R, D, T, x.data_ptr(), ldx, pi, out.data_ptr(), ldo)
    return out


def expert_combine(h, slots, weights=None, residual=None, out=None, stream=None):
    """out[t] = sum over j of weights[t,j] h[slots[t,j]] + residual[t]: h (R,D)
    of a 16-bit type, slots (T,k) int32 (outside 0 .. R - 1: nothing), weights
    (T,k) float32 or None for ones.  Without weights it is the gradient of
    expert_gather.  residual may be out."""
    on = _On(h, stream)
    dt = _dtype16(h, "h")
    if h.dim() != 2 or not isinstance(slots, on.torch.Tensor) or slots.dim() != 2:
        raise ValueError("h and slots must be matrices")
    R, D = h.shape
    T, k = slots.shape
    dtype = h.dtype
    ldh = on.mat(h, "h", dtype, R, D)
    ps = on.packed(slots, "slots", on.torch.int32, (T, k))
    pw = on.packed(weights, "weights", on.torch.float32, (T, k)) if weights is not None else 0
    pr = ldr = 0
    if residual is not None:
        ldr, pr = on.mat(residual, "residual", dtype, T, D), residual.data_ptr()
    out = on.new((T, D), dtype) if out is None else out
    ldo = on.mat(out, "out", dtype, T, D)
    on.call("expert_combine", dt, T, D, R, k, h.data_ptr(), ldh, ps, pw, pr, ldr, out.data_ptr(), ldo)
    return out


def expert_combine_backward(dout, h, slots, weights, dh=None, dweights=None, stream=None):
    """Gradients of expert_combine: (dh (R,D), dweights (T,k) float32).  Rows
    of dh that no slot names are not written."""
    on = _On(dout, stream)
    dt = _dtype16(dout, "dout")
    if dout.dim() != 2 or not isinstance(h, on.torch.Tensor) or h.dim() != 2 \
            or not isinstance(slots, on.torch.Tensor) or slots.dim() != 2:
        raise ValueError("dout, h and slots must be matrices")
    T, D = dout.shape
    R = h.shape[0]
    k = slots.shape[1]
    dtype = dout.dtype
    ldd = on.mat(dout, "dout", dtype, T, D)
    ldh = on.mat(h, "h", dtype, R, D)
    ps = on.packed(slots, "slots", on.torch.int32, (T, k))
    pw = on.packed(weights, "weights", on.torch.float32, (T, k))
    dh = on.new((R, D), dtype) if dh is None else dh
    ldg = on.mat(dh, "dh", dtype, R, D)
    dweights = on.new((T, k), on.torch.float32) if dweights is None else dweights
    pd = on.packed(dweights, "dweights", on.torch.float32, (T, k))
    on.call("expert_combine_backward", dt, T, D, R, k, dout.data_ptr(), ldd, h.data_ptr(), ldh, ps, pw,
            dh.data_ptr(), ldg, pd)
    return dh, dweights
