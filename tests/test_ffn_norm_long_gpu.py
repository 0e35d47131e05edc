"""The layer norm of long rows and of many rows on the GPU: no sum loses
digits as it gets longer.

Rows repeat eight values (and all rows are one), so that the 64-bit form of
the eight gives every mean and the tolerances of a short row.  None of the
values, squares or products is exact in binary32, and all of them have one
sign: what a chain of additions loses adds up."""
import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn
import _ffn_more_ref as more
import _ffn_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()
    yield
    torch.cuda.empty_cache()


def say(*what):
    print("[gpu]", *what, flush=True)


def eight(seed, dtype, lo=0.3, hi=1.1):
    g = torch.Generator().manual_seed(seed)
    return (lo + (hi - lo) * torch.rand(8, generator=g, dtype=torch.float64)).to(dtype)


def first_of_equal(t):
    """The first eight of values that repeat."""
    assert (t.view(-1, 8) == t.reshape(-1)[:8]).all()
    return t.reshape(-1)[:8][None]


# A row's sum goes through 3 additions within a piece of 8 values, 16 of a thread's pieces,
# a compensated sum of those (2 roundings), 6 additions between lanes and 16 between
# waves: at every length fewer than the 64 that the reference counts for a row of 8.
@pytest.mark.parametrize("N,dtype", [(20000, F32), (1 << 20, F32), (1 << 24, F32), (1 << 26, F32), ((1 << 31) - 4104, BF16)])
def test_long_rows(N, dtype):
    say("long row", N, dtype)
    x = eight(1, dtype)
    mean, rstd = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    y = tg.layer_norm(x.cuda().repeat(N // 8)[None], mean=mean, rstd=rstd)
    yr, ty, mu, r, tmu, tr, _, _ = more.layer_norm(x[None], None, None, 1e-5, dtype)
    ref.assert_near(mean, mu, tmu, "mean")
    ref.assert_near(rstd, r, tr, "rstd")
    ref.assert_near(first_of_equal(y), yr, ty, "y")


@pytest.mark.parametrize("N,dtype", [(8200, F32), (1 << 20, F32), (1 << 24, F32), (1 << 26, F32), ((1 << 30) - 8, BF16)])
def test_gradients_of_long_rows(N, dtype):
    say("long row's gradients", N, dtype)
    x, dy, w = eight(2, dtype), eight(3, dtype), eight(4, dtype)
    long = lambda t: t.cuda().repeat(N // 8)
    _, _, mu, r, _, _, _, _ = more.layer_norm(x[None], None, None, 1e-5, dtype)
    got = tg.layer_norm_backward(long(dy)[None], long(x)[None], long(w), mu.float().cuda(), r.float().cuda())
    want = more.layer_norm_backward(dy[None], x[None], w, 1e-5, None, dtype, dtype)
    for name, g in zip(("dx", "dweight", "dbias"), got):
        v, tol = want[name]
        ref.assert_near(first_of_equal(g), v.view(1, 8), tol.view(1, 8), name)


# The sums over M equal rows of 8 values: 512 workgroups of 8 rows a turn.  A
# thread's chain is at most 512 turns, then one addition per 512 turns; 8 row
# groups, 32 workgroups and 16 waves follow.
@pytest.mark.parametrize("M", [(1 << 20) + 5, (1 << 27) + 3])
def test_column_sums_of_many_rows(M):
    say("many rows", M)
    x, dy = eight(5, F32), eight(6, F32)
    _, _, mu, r, _, _, _, _ = more.layer_norm(x[None], None, None, 1e-5, F32)
    many = lambda t: t.cuda().repeat(M, 1)
    d = many(dy)
    mean, rstd = torch.full((M,), float(mu.float()), device="cuda"), torch.full((M,), float(r.float()), device="cuda")
    _, dw, db = tg.layer_norm_backward(d, many(x), None, mean, rstd, dx=d)
    # (Binary32 takes 3 roundings to dy h: the difference, h and the product.)
    h = (x.double() - mu.float().double()) * r.float().double()
    D = 512 + M / (512 * 8 * 512) + 8 + 32 + 16
    for name, got, v, each in (("dweight", dw, dy.double() * h, 3), ("dbias", db, dy.double(), 0)):
        want = M * v
        tol = M * v.abs() * (D + each) * more.U + ref.rounding(want, F32) * 1.001
        ref.assert_near(got, want, tol, name)
