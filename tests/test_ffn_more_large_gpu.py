"""The norm, the quantisation and the 4-bit products on arrays of more than
4 GiB, the longest rows, and graphs whose products split K.

What a large call gives at its ends is compared, bit for bit, with a small
call on a copy of those rows: the small sizes are held against 64-bit
references elsewhere."""
import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
GIB4 = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()
    yield
    torch.cuda.empty_cache()


@pytest.fixture
def tile():
    yield lambda size: ffn.set_tile(size, size)
    ffn.set_tile()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(seed, *shape):
    """Values of one tensor of this type, in place: no larger copies."""
    return torch.empty(*shape, dtype=BF16, device="cuda").normal_(generator=gen(seed))


def rand_mx(seed, rows, K):
    """Products of these are multiples of 1/16 of magnitudes about 6: every sum of up
    to 16384 fits 24 bits, and no order of additions changes it."""
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda").random_(0, 256, generator=gen(seed))
    s = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda").random_(126, 129, generator=gen(seed + 1))
    return q, s


@pytest.mark.parametrize("M,N", [(560001, 4096), (131101, 16640)])
def test_norm(M, N):
    print("[gpu] norm", M, N, flush=True)
    x, w, b = rand(0, M, N), rand(2, N), rand(3, N)
    dy = torch.empty_like(x).random_(-2, 3, generator=gen(1))
    assert x.numel() * 2 > GIB4
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    y = tg.layer_norm(x, w, b, mean=mean, rstd=rstd)
    dx, dw, db = tg.layer_norm_backward(dy, x, w, mean, rstd, residual=x)
    for part in (slice(0, 33), slice(M // 2, M // 2 + 33), slice(M - 33, M)):
        xs, ds = x[part].clone(), dy[part].clone()
        m, r = torch.empty(33, device="cuda"), torch.empty(33, device="cuda")
        assert torch.equal(y[part], tg.layer_norm(xs, w, b, mean=m, rstd=r))
        assert torch.equal(mean[part], m) and torch.equal(rstd[part], r)
        assert torch.equal(dx[part], tg.layer_norm_backward(ds, xs, w, m, r, residual=xs)[0])
    # The columns' sums in pieces, in 64 bits.  Those of dy are whole numbers: exact,
    # then rounded once.  Those of dy h, M terms of magnitude 2 at most on average,
    # meet in chains of at most M / 256 + 256 additions, each off by at most half a
    # step of the sum of magnitudes; the rounding to bfloat16 besides.
    want = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    for lo in range(0, M, 1 << 14):
        part = slice(lo, min(lo + (1 << 14), M))
        d = dy[part].double()
        want[1] += d.sum(0)
        want[0] += (d * ((x[part].double() - mean[part].double()[:, None]) * rstd[part].double()[:, None])).sum(0)
    assert torch.equal(db, want[1].to(BF16))
    tol = want[0].abs() * 2.0 ** -8 + (M / 256 + 256) * 2 * M * 2.0 ** -24
    assert ((dw.double() - want[0]).abs() <= tol).all()


@pytest.mark.parametrize("M,N", [(560001, 4096), (131101, 16640)])
def test_column_sums(M, N):
    """Of whole numbers, with mean 0 and rstd 1: exact sums, rounded once."""
    print("[gpu] column sums", M, N, flush=True)
    x, dy = (torch.empty(M, N, dtype=BF16, device="cuda").random_(-2, 3, generator=gen(i)) for i in range(2))
    _, dw, db = tg.layer_norm_backward(dy, x, None, torch.zeros(M, device="cuda"), torch.ones(M, device="cuda"))
    want = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    for lo in range(0, M, 1 << 14):
        d, v = dy[lo:lo + (1 << 14)].float(), x[lo:lo + (1 << 14)].float()
        want += torch.stack(((d * v).sum(0, dtype=torch.float64), d.sum(0, dtype=torch.float64)))
    assert torch.equal(dw, want[0].to(BF16)) and torch.equal(db, want[1].to(BF16))


def test_norm_of_the_longest_row():
    """+1 and -1 in turn: mean 0 and variance 1 without a rounding that matters to
    a bfloat16 (1 / sqrt(1 + 1e-5) is within 2^-9 of 1)."""
    N = (1 << 31) - 4104
    print("[gpu] norm 1", N, flush=True)
    x = torch.ones(N, dtype=BF16, device="cuda")
    x[1::2] = -1
    y = tg.layer_norm(x[None])
    assert torch.equal(y[0], x)


def test_gradients_of_the_widest_rows():
    """Gradients whose mean, and whose mean against the row, is 0: dx is dy, dweight dy times
    the row, all exact.  (The longest that the sums' workspace allows: more columns than
    one dispatch of the last step's workgroups.)"""
    N = (1 << 30) - 8
    print("[gpu] gradients 1", N, flush=True)
    four = lambda *v: torch.tensor(v, dtype=BF16, device="cuda").repeat(N // 4)
    x, dy = four(1, -1, 1, -1), four(1, 1, -1, -1)
    one = torch.ones(1, device="cuda")
    dx, dw, db = tg.layer_norm_backward(dy[None], x[None], None, 0 * one, one)
    assert torch.equal(dx[0], dy) and torch.equal(db, dy) and torch.equal(dw, four(1, -1, -1, 1))


def test_quantize():
    M, N = 524321, 16640
    print("[gpu] quantize", M, N, flush=True)
    x = rand(0, M, N)
    q, s, qt, st = tg.quantize_mxfp4(x, columns=True)
    assert q.numel() > GIB4 and qt.numel() > GIB4
    rows = slice(M - 65, M)
    few = tg.quantize_mxfp4(x[rows].clone())
    assert torch.equal(q[rows], few[0]) and torch.equal(s[rows], few[1])
    cols = slice(N - 64, N)
    few = tg.quantize_mxfp4(x[:, cols].clone(), rows=False, columns=True)
    assert torch.equal(qt[cols], few[0]) and torch.equal(st[cols], few[1])
    del x, qt, st, few
    # What elements stand for is quantised to the same values (a block whose largest
    # element is 3 takes half the scale, and twice the elements).
    back = tg.dequantize_mxfp4(q, s)
    del q, s
    assert torch.equal(tg.dequantize_mxfp4(*tg.quantize_mxfp4(back)), back)


@pytest.mark.parametrize("size", [64, 128, 256])
def test_products(size, tile):
    M, N, K = 70001, 32784, 256
    print("[gpu] product", M, N, K, size, flush=True)
    (a, sa), (b, sb) = rand_mx(0, M, K), rand_mx(2, N, K)
    bias, rows, cols = rand(4, N), slice(M - 130, M), slice(N - 264, N)
    tile(size)
    for act in ("none", "silu", "swiglu"):
        kept = torch.empty(M, N, dtype=BF16, device="cuda") if act == "silu" else None
        out = tg.gemm_mxfp4_epilogue(a, b, sa, sb, bias=bias, act=act, preact=kept)
        assert act == "swiglu" or out.numel() * 2 > GIB4
        few = tg.gemm_mxfp4_epilogue(a[rows].clone(), b, sa[rows].clone(), sb, bias=bias, act=act)
        assert torch.equal(out[rows], few), act
        if act != "swiglu":
            few = tg.gemm_mxfp4_epilogue(a, b[cols].clone(), sa, sb[cols].clone(), bias=bias[cols].clone(), act=act)
            assert torch.equal(out[:, cols], few), act
        if kept is not None:
            few = tg.gemm_mxfp4_epilogue(a[rows].clone(), b, sa[rows].clone(), sb, bias=bias)
            assert torch.equal(kept[rows], few)


@pytest.mark.parametrize("size", [16, 64, 128, 256])
def test_products_of_large_operands(size, tile):
    """A of more than 4 GiB, and the experts' weights."""
    M, N, K = 540001, 48, 16384
    print("[gpu] large operands", size, flush=True)
    a, sa = rand_mx(0, M, K)
    b, sb = rand_mx(2, N, K)
    assert a.numel() > GIB4
    tile(size)
    rows = slice(M - 37, M)
    assert torch.equal(tg.gemm_mxfp4_epilogue(a, b, sa, sb)[rows],
                       tg.gemm_mxfp4_epilogue(a[rows].clone(), b, sa[rows].clone(), sb))
    # The same bytes as 65 experts of 8208 x 16128 elements and a bit more.
    E, F, D = 65, 8208, 16128
    w, sw = a.view(-1)[:E * F * D // 2].view(E, F, D // 2), sa.view(-1)[:E * F * D // 32].view(E, F, D // 32)
    assert w.numel() > GIB4
    x, sx = rand_mx(4, 100, D)
    off = torch.tensor([0] * 63 + [0, 60, 90], dtype=torch.int32, device="cuda")
    out = tg.gemm_mxfp4_grouped(x, w, sx, sw, off)
    for e, part in ((63, slice(0, 60)), (64, slice(60, 90))):
        few = tg.gemm_mxfp4_epilogue(x[part].clone(), w[e].clone(), sx[part].clone(), sw[e].clone())
        assert torch.equal(out[part], few), e


@pytest.mark.parametrize("size", [64, 128, 256])
def test_grouped_rows(size, tile):
    """Outputs of more than 4 GiB by group, behind them rows of no group."""
    R, N, K = 70001, 32768, 256
    print("[gpu] grouped rows", size, flush=True)
    x, sx = rand_mx(0, R, K)
    w, sw = rand_mx(2, 2 * N, K)
    w, sw = w.view(2, N, -1), sw.view(2, N, -1)
    off = torch.tensor([0, 35000, R - 5], dtype=torch.int32, device="cuda")
    out = torch.full((R, N), 3.0, dtype=BF16, device="cuda")
    tile(size)
    tg.gemm_mxfp4_grouped(x, w, sx, sw, off, out=out)
    assert out.numel() * 2 > GIB4 and (out[R - 5:] == 3).all()
    part = slice(R - 105, R - 5)
    assert torch.equal(out[part], tg.gemm_mxfp4_epilogue(x[part].clone(), w[1], sx[part].clone(), sw[1]))


def test_graphs_that_split_k():
    """Two graphs, each with a workspace of its own pool, replayed in turn with
    eager calls between them."""
    M, N, K = 48, 512, 16384
    assert ffn.lib().tgemm_mxfp4_workspace_bytes(M, N, K) > 0
    x = [rand(i, M, K) for i in range(2)]
    b, sb = rand_mx(5, N, K)
    graphs, outs = [], []
    for i in range(2):
        outs.append(torch.zeros(M, N, dtype=BF16, device="cuda"))
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[i]):
            a, sa = tg.quantize_mxfp4(x[i])
            tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="gelu", out=outs[i])
    for turn in range(4):
        for i in range(2):
            x[i].normal_(generator=gen(10 + 2 * turn + i))
            outs[i].zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            a, sa = tg.quantize_mxfp4(x[i])
            assert torch.equal(outs[i], tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="gelu"))
