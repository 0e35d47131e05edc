"""The layer norm and the MXFP4 operators on the host: bad arguments are
refused with the documented status before any device is touched.  No test here
launches a kernel."""
import math
import os
import re
import subprocess

import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn

P = [0x10000 + (i << 36) for i in range(1, 14)]   # plausible device addresses, 64 GiB apart; a refused call uses none
BIG = (1 << 31) - 4096


def refused(name, code, word, **fields):
    rc = getattr(ffn.lib(), name)(ffn.args(name, **fields), None)
    assert rc == code, (rc, ffn.last_error())
    assert word in ffn.last_error(), ffn.last_error()


def norm(**kw):
    return {**dict(dtype=0, wdtype=0, M=16, N=64, x=P[0], ldx=64, weight=P[1], bias=P[2], eps=1e-5, y=P[3], ldy=64,
                   mean=P[4], rstd=P[5]), **kw}


@pytest.mark.parametrize("fields,code,word", [
    (norm(dtype=3), tg.EINVAL, "element type"), (norm(dtype=-1), tg.EINVAL, "element type"),
    (norm(wdtype=1), tg.EINVAL, "weight's type"), (norm(dtype=2, wdtype=0), tg.EINVAL, "weight's type"),
    (norm(M=-1), tg.EINVAL, "negative"), (norm(M=BIG), tg.ETOOBIG, "sizes"), (norm(N=BIG), tg.ETOOBIG, "sizes"),
    (norm(N=0), tg.EINVAL, "at least 8"), (norm(N=60), tg.EALIGN, "multiple of 8"), (norm(eps=-1e-9), tg.EINVAL, "eps"),
    (norm(eps=math.nan), tg.EINVAL, "eps"), (norm(eps=math.inf), tg.EINVAL, "eps"), (norm(eps=1e39), tg.EINVAL, "eps"),
    (norm(x=0), tg.EINVAL, "x is NULL"), (norm(y=0), tg.EINVAL, "y is NULL"), (norm(x=P[0] + 8), tg.EALIGN, "x is not"),
    (norm(ldx=56), tg.EINVAL, "stride of x"), (norm(ldx=68), tg.EALIGN, "stride of x"), (norm(ldy=32), tg.EINVAL, "stride of y"),
    (norm(ldx=1 << 31), tg.ETOOBIG, "stride of x"), (norm(weight=P[1] + 4), tg.EALIGN, "weight"),
    (norm(mean=P[4] + 2), tg.EALIGN, "mean"), (norm(y=P[0] + 16), tg.EINVAL, "y overlaps x"),
    (norm(y=P[0], ldy=72), tg.EINVAL, "y overlaps x"), (norm(mean=P[3]), tg.EINVAL, "overlaps"),
    (norm(rstd=P[1]), tg.EINVAL, "rstd overlaps weight"),
])
def test_layer_norm_refuses(fields, code, word):
    refused("layer_norm", code, word, **fields)


def nback(**kw):
    return {**dict(dtype=0, wdtype=2, M=100, N=64, dy=P[0], ldd=64, x=P[1], ldx=64, weight=P[2], mean=P[3], rstd=P[4],
                   residual=P[5], ldr=64, dx=P[6], ldo=64, dweight=P[7], dbias=P[8], workspace=P[9],
                   workspace_bytes=1 << 24), **kw}


@pytest.mark.parametrize("fields,code,word", [
    (nback(dtype=5), tg.EINVAL, "element type"), (nback(wdtype=1), tg.EINVAL, "weight's type"),
    (nback(N=4), tg.EINVAL, "at least 8"), (nback(dy=0), tg.EINVAL, "dy is NULL"), (nback(x=0), tg.EINVAL, "x is NULL"),
    (nback(mean=0), tg.EINVAL, "mean is NULL"), (nback(rstd=0), tg.EINVAL, "rstd is NULL"), (nback(dx=0), tg.EINVAL, "dx is NULL"),
    (nback(workspace=0), tg.EINVAL, "workspace is NULL"), (nback(workspace=P[9] + 4), tg.EALIGN, "workspace"),
    (nback(workspace_bytes=64), tg.EINVAL, "workspace bytes"), (nback(workspace=P[1]), tg.EINVAL, "overlaps"),
    (nback(dx=P[0] + 16), tg.EINVAL, "dx overlaps dy"), (nback(dx=P[5], ldo=72), tg.EINVAL, "dx overlaps residual"),
    (nback(dweight=P[6]), tg.EINVAL, "overlaps"), (nback(dbias=P[7]), tg.EINVAL, "dweight overlaps dbias"),
    (nback(ldd=60), tg.EINVAL, "stride of dy"), (nback(ldr=32), tg.EINVAL, "stride of residual"),
    (nback(dweight=P[7] + 8), tg.EALIGN, "dweight"),
])
def test_layer_norm_backward_refuses(fields, code, word):
    refused("layer_norm_backward", code, word, **fields)


def quant(**kw):
    return {**dict(dtype=0, M=100, N=64, x=P[0], ldx=64, q=P[1], ldq=32, scales=P[2], qt=P[3], ldqt=64, scalest=P[4]), **kw}


@pytest.mark.parametrize("fields,code,word", [
    (quant(dtype=3), tg.EINVAL, "element type"), (quant(N=40, ldx=40), tg.EALIGN, "multiple of 32"),
    (quant(N=36, q=0, scales=0, ldx=40), tg.EALIGN, "multiple of 8"), (quant(x=0), tg.EINVAL, "x is NULL"),
    (quant(q=0), tg.EINVAL, "q is NULL"), (quant(scales=0), tg.EINVAL, "scales is NULL"),
    (quant(qt=0), tg.EINVAL, "qt is NULL"), (quant(scalest=0), tg.EINVAL, "scalest is NULL"),
    (quant(q=0, scales=0, qt=0, scalest=0), tg.EINVAL, "q is NULL"), (quant(ldq=16), tg.EINVAL, "stride of q"),
    (quant(ldq=40), tg.EALIGN, "stride of q"), (quant(ldqt=72), tg.EALIGN, "stride of qt"),
    (quant(ldqt=48), tg.EINVAL, "stride of qt"), (quant(q=P[1] + 8), tg.EALIGN, "q is not"),
    (quant(q=P[0]), tg.EINVAL, "q overlaps x"), (quant(scalest=P[2]), tg.EINVAL, "overlaps"),
    (quant(ldx=32), tg.EINVAL, "stride of x"), (quant(M=BIG), tg.ETOOBIG, "sizes"),
])
def test_quantize_refuses(fields, code, word):
    refused("quantize_mxfp4", code, word, **fields)


def dequant(**kw):
    return {**dict(dtype=0, M=8, N=64, q=P[0], ldq=32, scales=P[1], out=P[2], ldo=64), **kw}


@pytest.mark.parametrize("fields,code,word", [
    (dequant(dtype=4), tg.EINVAL, "element type"), (dequant(N=48), tg.EALIGN, "multiple of 32"),
    (dequant(q=0), tg.EINVAL, "q is NULL"), (dequant(scales=0), tg.EINVAL, "scales is NULL"),
    (dequant(out=0), tg.EINVAL, "out is NULL"), (dequant(ldq=24), tg.EINVAL, "stride of q"),
    (dequant(ldq=40), tg.EALIGN, "stride of q"), (dequant(out=P[0]), tg.EINVAL, "out overlaps q"),
])
def test_dequantize_refuses(fields, code, word):
    refused("dequantize_mxfp4", code, word, **fields)


def mx(**kw):
    return {**dict(dtype=0, M=16, N=32, K=64, A=P[0], lda=32, scale_A=P[1], B=P[2], ldb=32, scale_B=P[3], C=P[4], ldc=32), **kw}


@pytest.mark.parametrize("fields,code,word", [
    (mx(dtype=2), tg.EINVAL, "element type"), (mx(M=-1), tg.EINVAL, "negative"), (mx(N=BIG), tg.ETOOBIG, "sizes"),
    (mx(K=48), tg.EALIGN, "multiple of 32"), (mx(act=7), tg.EINVAL, "activation"),
    (mx(act=5, N=24, ldc=16), tg.EALIGN, "multiple of 16"), (mx(N=36, ldc=40), tg.EALIGN, "row length of C"),
    (mx(A=0), tg.EINVAL, "A is NULL"), (mx(scale_A=0), tg.EINVAL, "scale_A is NULL"), (mx(B=0), tg.EINVAL, "B is NULL"),
    (mx(scale_B=0), tg.EINVAL, "scale_B is NULL"), (mx(C=0), tg.EINVAL, "C is NULL"),
    (mx(A=P[0] + 8), tg.EALIGN, "A is not"), (mx(lda=16), tg.EINVAL, "stride of A"), (mx(lda=40), tg.EALIGN, "stride of A"),
    (mx(ldb=56), tg.EALIGN, "stride of B"), (mx(ldc=24), tg.EINVAL, "stride of C"), (mx(C=P[0]), tg.EINVAL, "C overlaps A"),
    (mx(C=P[3]), tg.EINVAL, "C overlaps scale_B"), (mx(residual=P[4] + 16, ldr=32), tg.EINVAL, "C overlaps residual"),
    (mx(preact=P[5], ldp=16), tg.EINVAL, "stride of preact"), (mx(lda=1 << 23), tg.ETOOBIG, "A too large"),
    (mx(ldb=1 << 23), tg.ETOOBIG, "B too large"), (mx(act=5, N=1 << 23, ldb=512, ldc=1 << 22), tg.ETOOBIG, "B too large"),
    (mx(bias=P[6] + 2), tg.EALIGN, "bias"),
])
def test_mx_epilogue_refuses(fields, code, word):
    refused("gemm_mxfp4_epilogue", code, word, **fields)


def grp(**kw):
    return {**dict(dtype=0, R=64, N=32, K=64, groups=4, offsets=P[5], src_rows=64, A=P[0], lda=32, scale_A=P[1], B=P[2],
                   ldb=32, stride_b=1024, scale_B=P[3], stride_sb=64, C=P[4], ldc=32), **kw}


@pytest.mark.parametrize("fields,code,word", [
    (grp(dtype=2), tg.EINVAL, "element type"), (grp(K=40), tg.EALIGN, "multiple of 32"), (grp(offsets=0), tg.EINVAL, "offsets is NULL"),
    (grp(offsets=P[5] + 2), tg.EALIGN, "offsets"), (grp(rows=P[6] + 1), tg.EALIGN, "rows"),
    (grp(stride_b=-16), tg.EINVAL, "stride_b"), (grp(stride_sb=-1), tg.EINVAL, "stride_sb"),
    (grp(stride_b=8), tg.EALIGN, "stride_b"), (grp(stride_b=1 << 41), tg.ETOOBIG, "stride_b"),
    (grp(groups=65537), tg.ETOOBIG, "65536"), (grp(C=P[2] + 3 * 1024), tg.EINVAL, "C overlaps B"),
    (grp(C=P[3] + 3 * 64), tg.EINVAL, "C overlaps B or its scales"), (grp(rows=P[6], src_rows=1 << 26), tg.ETOOBIG, "A too large"),
    (grp(scale_A=0), tg.EINVAL, "scale_A is NULL"), (grp(act=6, N=40, ldc=24), tg.EALIGN, "multiple of 16"),
    (grp(preact=P[7], ldp=8), tg.EINVAL, "stride of preact"),
])
def test_mx_grouped_refuses(fields, code, word):
    refused("gemm_mxfp4_grouped", code, word, **fields)


def deep(**kw):
    """A call whose K is split."""
    return mx(M=64, K=8192, lda=4096, ldb=4096, workspace_bytes=1 << 22, **kw)


@pytest.mark.parametrize("fields,code,word", [
    (deep(workspace=P[8] + 4), tg.EALIGN, "workspace"), (deep(workspace=P[0] + 4096), tg.EINVAL, "workspace overlaps A"),
    (deep(workspace=P[3]), tg.EINVAL, "workspace overlaps scale_B"), (deep(workspace=P[4]), tg.EINVAL, "C overlaps workspace"),
])
def test_mx_split_refuses(fields, code, word):
    refused("gemm_mxfp4_epilogue", code, word, **fields)


def test_workspace_sizes():
    mxw, norm_w = ffn.lib().tgemm_mxfp4_workspace_bytes, ffn.lib().tgemm_layer_norm_backward_workspace_bytes
    assert mxw(64, 32, 8192) == 4 * 64 * 32 * 4
    assert mxw(48, 8192, 28672) == 2 * 48 * 8192 * 4
    assert mxw(16, 32, 8192) == 0                    # few rows split K by themselves
    assert mxw(64, 32, 4096) == 0                    # not deep enough
    assert mxw(1024, 1024, 1 << 20) == 0             # enough tiles without
    assert mxw(0, 32, 8192) == mxw(64, -8, 8192) == mxw(64, 1 << 31, 8192) == mxw(64, 32, 1 << 31) == 0
    assert norm_w(1, 4096) == 2 * 4096 * 4
    assert norm_w(8192, 4096) == 256 * 2 * 4096 * 4
    assert norm_w(128, 16384) == (256 + 2 * 2 * 16384) * 4      # two steps: a pair a row, a pair of sums a 64 rows
    assert norm_w(0, 64) == norm_w(-1, 64) == norm_w(64, 0) == norm_w(1 << 31, 64) == 0


def test_the_kernels_keep_their_accumulators_in_registers(tmp_path):
    """No kernel of these operators uses scratch memory."""
    tools = "/opt/rocm/lib/llvm/bin"
    if not os.path.exists(os.path.join(tools, "llvm-readelf")):
        pytest.skip("no LLVM tools")
    so = tmp_path / "lib.so"
    so.write_bytes(open(ffn.LIB_PATH, "rb").read())
    subprocess.run([os.path.join(tools, "llvm-objdump"), "--offloading", str(so)], capture_output=True, check=True,
                   cwd=tmp_path)
    seen = 0
    for f in tmp_path.glob("lib.so.*gfx950*"):
        notes = subprocess.run([os.path.join(tools, "llvm-readelf"), "--notes", str(f)], capture_output=True, text=True,
                               check=True).stdout
        for name, size in re.findall(r"\.name:\s+(\S+).*?\.private_segment_fixed_size:\s+(\d+)", notes, re.S):
            if re.search(r"(mx_\w+|norm\w*|quant\w*)_kernel", name):
                seen += 1
                assert int(size) == 0, name
    assert seen > 100


def test_nothing_to_do_needs_no_device():
    call = lambda name, **f: getattr(ffn.lib(), name)(ffn.args(name, **f), None)
    assert call("layer_norm", **norm(M=0, x=0, y=0)) == tg.OK
    assert call("layer_norm_backward", **nback(M=0, dweight=0, dbias=0)) == tg.OK
    assert call("quantize_mxfp4", **quant(M=0)) == call("dequantize_mxfp4", **dequant(M=0)) == tg.OK
    assert call("gemm_mxfp4_epilogue", **mx(M=0)) == call("gemm_mxfp4_epilogue", **mx(N=0)) == tg.OK
    assert call("gemm_mxfp4_grouped", **grp(R=0)) == call("gemm_mxfp4_grouped", **grp(groups=0)) == tg.OK


def test_the_binding_refuses_what_is_not_on_a_gpu():
    x, b = torch.zeros(8, 32), torch.zeros(8, 16, dtype=torch.uint8)
    s = torch.zeros(8, 1, dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: tg.layer_norm(x), lambda: tg.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
              lambda: tg.quantize_mxfp4(x), lambda: tg.dequantize_mxfp4(b, s), lambda: tg.gemm_mxfp4_epilogue(b, b, s, s),
              lambda: tg.gemm_mxfp4_grouped(b, b[None], s, s[None], off)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError, match="dtype"):
        tg.dequantize_mxfp4(b, s, dtype=torch.float64)
    with pytest.raises(ValueError, match="act"):
        tg.gemm_mxfp4_epilogue(b, b, s, s, act="tanh")
