"""MXFP4 products by the library's own choice of a kernel, each kernel at sizes
that take it (test_ffn_mx_choice_host.py holds the library to that), dense and
by group, against the 64-bit form at rows around every border."""
import math

import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn
import _ffn_mx_choice as mx
import _ffn_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()
    yield
    torch.cuda.empty_cache()


def rand(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def rand_mx(seed, rows, K, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    s = torch.randint(124 - shift, 131 - shift, (rows, K // 32), generator=g, dtype=torch.uint8, device="cuda")
    return q, s


def values(q, s):
    """What they stand for, in 64 bits (binary32 holds each)."""
    return tg.dequantize_mxfp4(q, s, dtype=F32).double()


def some_rows(lo, hi):
    """Rows around the ends and around the borders of 16, 64, 128 and 256."""
    at = [lo + o for o in (0, 1, 15, 16, 63, 64, 127, 128, 255, 256, (hi - lo) // 2)] + [hi - 1 - o for o in (0, 1, 17, 65)]
    return torch.tensor(sorted({r for r in at if lo <= r < hi}), device="cuda")


def check(out, z, rows, x, b, bias, act, residual, dtype, what):
    yr, ty, zr, tz = (t.cpu() for t in ref.epilogue(x, b.t().contiguous(), bias, act, residual, dtype))
    ref.assert_near(out[rows], yr, ty, what)
    if z is not None:
        ref.assert_near(z[rows], zr, tz, "preact of " + what)


@pytest.mark.parametrize("kernel,M,N,K,act,bias,residual,preact", mx.DENSE)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_dense(kernel, M, N, K, act, bias, residual, preact, dtype):
    print("[gpu]", kernel, M, N, K, act, dtype, flush=True)
    F = N // 2 if act in ref.GATED else N
    a, sa = rand_mx(1, M, K)
    b, sb = rand_mx(2, N, K, int(math.log2(K) / 2) + 2)          # sums of about unit size
    bs = rand(3, N, dtype=dtype) if bias else None
    rs = rand(4, M, F, dtype=dtype) if residual else None
    z = torch.full((M, N), 7.0, dtype=dtype, device="cuda") if preact else None
    out = torch.full((M, F), 9.0, dtype=dtype, device="cuda")
    tg.gemm_mxfp4_epilogue(a, b, sa, sb, bias=bs, act=act, residual=rs, preact=z, out=out)
    rows = some_rows(0, M)
    check(out, z, rows, values(a, sa)[rows], values(b, sb), bs, act, None if rs is None else rs[rows], dtype, f"{M}x{N}x{K}")


@pytest.mark.parametrize("kernel,R,E,N,K,act,bias,preact", mx.GROUPED)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped(kernel, R, E, N, K, act, bias, preact, gather, dtype):
    print("[gpu]", kernel, R, E, N, K, act, gather, dtype, flush=True)
    F = N // 2 if act in ref.GATED else N
    g = torch.Generator().manual_seed(R)
    off = torch.cat((torch.zeros(1), torch.randint(0, R, (E - 1,), generator=g).sort().values, torch.tensor([R]))).int()
    S = R // 2 + 3 if gather else R
    a, sa = rand_mx(1, S, K)
    b, sb = rand_mx(2, E * N, K, int(math.log2(K) / 2) + 2)
    b, sb = b.view(E, N, -1), sb.view(E, N, -1)
    src = torch.randint(0, S, (R,), generator=g, dtype=torch.int32).cuda() if gather else None
    bs = rand(3, E, N, dtype=dtype) if bias else None
    z = torch.full((R, N), 7.0, dtype=dtype, device="cuda") if preact else None
    out = torch.full((R, F), 9.0, dtype=dtype, device="cuda")
    tg.gemm_mxfp4_grouped(a, b, sa, sb, off.cuda(), rows=src, bias=bs, act=act, preact=z, out=out)
    av = values(a, sa)
    for e in range(E):
        rows = some_rows(int(off[e]), int(off[e + 1]))
        if len(rows):
            x = av[rows if src is None else src[rows].long()]
            check(out, z, rows, x, values(b[e], sb[e]), None if bs is None else bs[e], act, None, dtype, f"group {e}")
