"""The feed-forward products on the GPU against their plain 64-bit forms:
every layout, tile and activation, odd sizes, strides, empty groups, indexes
outside the operand, gradients, graphs, streams.  Tolerances are half a step
of the output type plus the error that 32-bit sums of that length may have
(_ffn_ref.py)."""
import math
import threading

import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn
import _ffn_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
LAYOUTS = ["nt", "nn", "tn", "tt"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()


@pytest.fixture
def tile():
    yield ffn.set_tile
    ffn.set_tile()


def rand(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def stored(x, transposed):
    """x (CPU) on the GPU, as the transpose of a row-major array if asked."""
    return x.t().contiguous().cuda().t() if transposed else x.cuda()


def say(*what):
    print("[gpu]", *what, flush=True)


def run_epilogue(M, N, K, dtype, layout, act, bias=True, residual=True, preact=True, seed=0):
    F = N // 2 if act in ref.GATED else N
    a = rand(seed, M, K, dtype=dtype)
    b = rand(seed + 1, K, N, dtype=dtype, scale=1 / math.sqrt(max(K, 1)))
    bs = rand(seed + 2, N, dtype=dtype) if bias else None
    rs = rand(seed + 3, M, F, dtype=dtype) if residual else None
    z = torch.full((M, N), 7.0, dtype=dtype, device="cuda") if preact else None
    say("epilogue", M, N, K, dtype, layout, act, bias, residual, preact)
    y = tg.gemm_epilogue(stored(a, layout[0] == "t"), stored(b, layout[1] == "t"), bias=None if bs is None else bs.cuda(),
                         act=act, residual=None if rs is None else rs.cuda(), preact=z)
    torch.cuda.synchronize()
    yr, ty, zr, tz = ref.epilogue(a, b, bs, act, rs, dtype)
    assert y.dtype == dtype
    ref.assert_near(y, yr, ty, "out")
    if preact:
        ref.assert_near(z, zr, tz, "preact")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 264, 1000), (3, 40, 64), (16, 16, 72), (17, 136, 520), (33, 48, 136),
                                   (64, 72, 2056)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_few_rows(dtype, M, N, K, act):
    run_epilogue(M, N, K, dtype, "nt", act, seed=M + N + K)


@pytest.mark.parametrize("act", ref.GATED)
@pytest.mark.parametrize("M,N,K", [(1, 16, 8), (5, 80, 200), (31, 48, 1032), (50, 1040, 328)])
def test_few_rows_gated(act, M, N, K):
    run_epilogue(M, N, K, BF16, "nt", act, residual=M % 2 == 1, seed=M)
    run_epilogue(M, N, K, F16, "nt", act, bias=False, preact=False, seed=M + 9)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [(256, 256), (256, 192), (128, 128), (64, 64)])
def test_tiles_and_layouts(layout, size, tile):
    if size == (256, 192) and layout[1] == "n":
        pytest.skip("256 x 192 tiles take B stored N x K")
    tile(*size)
    for i, (M, N, K) in enumerate([(296, 264, 136), (72, 520, 72), (8, 8, 200)]):
        run_epilogue(M, N, K, BF16 if i != 1 else F16, layout, ACTS[(i + len(layout)) % 5], bias=i != 1,
                     residual=i != 2, preact=i != 0, seed=i)


@pytest.mark.parametrize("layout", ["nt", "nn"])
@pytest.mark.parametrize("size", [256, 128, 64])
@pytest.mark.parametrize("act", ref.GATED)
def test_tiles_gated(layout, size, act, tile):
    tile(size, size)
    run_epilogue(300, 528, 136, BF16, layout, act, seed=1)
    run_epilogue(67, 272, 72, F16, layout, act, bias=False, residual=False, preact=False, seed=2)
    run_epilogue(9, 16, 200, BF16, layout, act, seed=3)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_activations_on_a_large_tile(act, dtype, tile):
    tile(256, 256)
    run_epilogue(256, 256, 64, dtype, "nt", act, seed=4)


def test_chosen_tiles():
    """Sizes that take each kernel by the library's own choice."""
    for M, N, K in [(65, 512, 256), (400, 1000, 264), (2048, 2048, 128), (1030, 4104, 72)]:
        run_epilogue(M, N, K, BF16, "nt", "gelu_tanh", seed=M)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M,N,K,act", [(1, 24, 4168, "gelu"), (72, 264, 4200, "silu"), (40, 1040, 2056, "none"),
                                       (553, 136, 2568, "relu"), (130, 272, 8200, "gelu_tanh")])
def test_split_k(layout, M, N, K, act):
    if layout[0] == "t":
        M = (M + 7) // 8 * 8  # rows of an A stored K x M are 16-byte multiples
    assert ffn.lib().tgemm_epilogue_workspace_bytes(layout[0] == "t", layout[1] == "t", M, N, K) > 0
    run_epilogue(M, N, K, BF16, layout, act, seed=M)
    run_epilogue(M, N, K, F16, layout, act, bias=False, residual=False, preact=False, seed=M + 9)


@pytest.mark.parametrize("layout", ["nt", "nn"])
@pytest.mark.parametrize("act", ref.GATED)
@pytest.mark.parametrize("M,N,K", [(3, 16, 4168), (100, 1040, 2568), (989, 352, 2056)])
def test_split_k_gated(layout, act, M, N, K):
    assert ffn.lib().tgemm_epilogue_workspace_bytes(0, layout[1] == "t", M, N, K) > 0
    run_epilogue(M, N, K, BF16, layout, act, seed=M)
    run_epilogue(M, N, K, F16, layout, act, bias=False, residual=False, preact=False, seed=M + 9)


def test_split_k_workspaces():
    """The sums stay within the bytes asked for; with a byte less K is not
    split; calls of two streams and a replayed graph have the same bits."""
    M, N, K = 100, 264, 4168
    a, b, r, bias = rand(1, M, K).cuda(), rand(2, N, K, scale=0.02).cuda(), rand(3, M, N).cuda(), rand(4, N).cuda()
    need = ffn.lib().tgemm_epilogue_workspace_bytes(0, 1, M, N, K)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")

    def run(**kw):
        return tg.gemm_epilogue(a, b.t(), bias=bias, act="silu", residual=r, **kw)

    want = run()
    assert torch.equal(run(workspace=ws[:need]), want)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 77).all()) and not bool((ws[:need] == 77).all())
    ws.fill_(77)
    short = run(workspace=ws[:need - 1])
    torch.cuda.synchronize()
    assert bool((ws == 77).all())
    for y in (want, short):
        yr, ty, _, _ = ref.epilogue(a.cpu(), b.t().cpu(), bias.cpu(), "silu", r.cpu(), BF16)
        ref.assert_near(y, yr, ty)
    out = r.clone()
    assert torch.equal(tg.gemm_epilogue(a, b.t(), bias=bias, act="silu", residual=out, out=out), want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [run(stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    for i in range(3):
        a.copy_(rand(20 + i, M, K))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
    with pytest.raises(tg.TgemmError, match="overlaps"):
        run(workspace=b.view(torch.uint8).view(-1))  # (a's bytes are fewer than the sums take)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M", [8, 200])
def test_empty_k(layout, M):
    run_epilogue(M, 24, 0, BF16, layout, "gelu", seed=5)


def test_strides_and_bytes_around_are_left(tile):
    """Operands inside larger arrays filled with NaN (which a read past a row's
    end would bring in), outputs inside arrays that must keep what is around."""
    for size in (16, 64, 128, 256):
        tile(size, size)
        for act, N in (("silu", 136), ("swiglu", 272)):
            M, K = 37, 200
            F = N // 2 if act in ref.GATED else N
            nan = float("nan")

            def inside(x, rows=3, cols=24):
                big = torch.full((x.shape[0] + 2 * rows, x.shape[1] + 2 * cols), nan, dtype=x.dtype, device="cuda")
                view = big[rows:rows + x.shape[0], cols:cols + x.shape[1]]
                view.copy_(x)
                return view, big

            a, b = rand(1, M, K), rand(2, N, K, scale=0.1)
            r, bias = rand(3, M, F), rand(4, N)
            av, _ = inside(a)
            bv, _ = inside(b)
            rv, _ = inside(r)
            out, big = inside(torch.zeros(M, F, dtype=BF16))
            z, zbig = inside(torch.zeros(M, N, dtype=BF16))
            say("strides", size, act)
            tg.gemm_epilogue(av, bv.t(), bias=bias.cuda(), act=act, residual=rv, preact=z, out=out)
            torch.cuda.synchronize()
            yr, ty, zr, tz = ref.epilogue(a, b.t(), bias, act, r, BF16)
            ref.assert_near(out, yr, ty, "out")
            ref.assert_near(z, zr, tz, "preact")
            for t, n in ((big, M * F), (zbig, M * N)):
                assert int(torch.isnan(t).sum()) == t.numel() - n, "bytes around the output were written"


def test_residual_may_be_the_output(tile):
    for size in (16, 128):
        tile(size, size)
        a, b, r = rand(1, 40, 72), rand(2, 48, 72), rand(3, 40, 48)
        out = r.cuda()
        tg.gemm_epilogue(a.cuda(), b.cuda().t(), act="relu", residual=out, out=out)
        yr, ty, _, _ = ref.epilogue(a, b.t(), None, "relu", r, BF16)
        ref.assert_near(out, yr, ty)


def test_special_values_stay_in_their_row(tile):
    for size in (16, 64, 256):
        tile(size, size)
        for act in ACTS:
            a, b = rand(1, 48, 136), rand(2, 64, 136, scale=0.1)
            a[5, 100] = float("nan")
            a[9, 3] = float("inf")
            b[7] = 0
            y = tg.gemm_epilogue(a.cuda(), b.cuda().t(), act=act).cpu()
            torch.cuda.synchronize()
            clean = [i for i in range(48) if i not in (5, 9)]
            yr, ty, _, _ = ref.epilogue(a[clean], b.t(), None, act, None, BF16)
            ref.assert_near(y[clean], yr, ty, act)
            assert torch.isnan(y[5]).all()
            # inf * 0 = NaN in column 7; elsewhere the activation of an infinity
            assert torch.isnan(y[9, 7])
            want = ref.layer(a[9:10].double() @ b.t().double(), act)[0]
            if act in ("none", "relu"):
                assert torch.equal(torch.isinf(y[9].double()), torch.isinf(want))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_activation_values_over_their_range(act, dtype):
    """Every size of argument up to the type's largest, through a product with
    the identity."""
    top = 60000.0 if dtype == F16 else 1e38
    mag = torch.logspace(-6, math.log10(top), 500, dtype=torch.float64)
    x = torch.cat([mag, -mag]).to(dtype).view(125, 8)
    eye = torch.eye(8, dtype=dtype)
    y = tg.gemm_epilogue(x.cuda(), eye.cuda().t(), act=act).cpu()
    z = x.double()
    yr = ref.layer(z, act)
    # Far down the negative tail the value vanishes: the kernel's exponential
    # ends at 2^-126, where |z| is below 2^7.
    tol = ref.rounding(yr, dtype) * 1.01 + ref.VALUE * yr.abs() + 2.0 ** -118
    if act in ("gelu", "gelu_tanh", "silu"):
        tol = tol + torch.where(z < 0, 2.0 ** -17 * z.abs() * yr.abs() * 8, torch.zeros_like(z))
    ref.assert_near(y, yr, tol, act)


# --------------------------------------------------------------------------
# The epilogue's backward pass
# --------------------------------------------------------------------------
def grad_formula(dy, z, act):
    z = z.double().detach().requires_grad_()
    ref.layer(z, act).backward(dy.double())
    return z.grad


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu"])
def test_reference_gradient_against_differences(act):
    z = torch.linspace(-4, 4, 64, dtype=torch.float64).view(4, 16) + 0.01
    dy = rand(1, 4, 8 if act in ref.GATED else 16).double()
    g, h = grad_formula(dy, z, act), 1e-5
    for i in range(4):
        for j in range(16):
            d = torch.zeros_like(z)
            d[i, j] = h
            num = ((ref.layer(z + d, act) - ref.layer(z - d, act)) * dy).sum() / (2 * h)
            assert abs(num - g[i, j]) < 1e-7


# The derivatives' slopes are at most 1.13, like the activations'; their
# kernels' values are within 2^-17 relative to the terms they add.
def grad_tolerance(dy, z, act, dz):
    dy = dy.double().abs()
    if act in ref.GATED:
        g, u = z.double().chunk(2, dim=1)
        e = torch.cat((dy * u.abs() * 2.0 ** -15, dy * g.abs() * 2.0 ** -15), 1)
    else:
        e = dy * 2.0 ** -15 if act not in ("none", "relu") else torch.zeros_like(dz)
    return e


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,F", [(1, 8), (63, 264), (200, 40), (700, 1000)])
def test_epilogue_backward(act, dtype, M, F):
    N = 2 * F if act in ref.GATED else F
    z, dy = rand(1, M, N, dtype=dtype, scale=2.0), rand(2, M, F, dtype=dtype)
    say("epilogue_backward", act, dtype, M, F)
    dz, dbias = tg.epilogue_backward(dy.cuda(), z.cuda() if act != "none" else None, act)
    torch.cuda.synchronize()
    want = grad_formula(dy, z, act)
    e = grad_tolerance(dy, z, act, want)
    ref.assert_near(dz, want, e + ref.rounding(want, dtype) * 1.01, "dz")
    s = want.sum(0)
    ref.assert_near(dbias, s, e.sum(0) + (M + 16) * 2.0 ** -24 * want.abs().sum(0) + ref.rounding(s, dtype) * 1.01,
                    "dbias")


def test_epilogue_backward_groups():
    for counts in ([5, 0, 64, 65, 1, 0, 130], [0, 0, 0], [300], [1] * 70):
        off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
        M, used = int(off[-1]) + 7, int(off[-1])
        for act, F in (("silu", 72), ("swiglu", 264), ("none", 24)):
            N = 2 * F if act in ref.GATED else F
            z, dy = rand(1, M, N), rand(2, M, F)
            buf = torch.full((M, N), 3.0, dtype=BF16, device="cuda")
            ws = torch.full((1 << 20,), float("nan"), device="cuda")
            say("groups", counts[:8], act)
            dz, db = tg.epilogue_backward(dy.cuda(), z.cuda(), act, offsets=off.cuda(), dz=buf, workspace=ws)
            torch.cuda.synchronize()
            want = grad_formula(dy, z, act)
            e = grad_tolerance(dy, z, act, want)
            ref.assert_near(dz[:used], want[:used], (e + ref.rounding(want, BF16) * 1.01)[:used], "dz")
            assert (dz[used:].cpu() == 3.0).all(), "rows behind the last group were written"
            for g, n in enumerate(counts):
                r = slice(int(off[g]), int(off[g]) + n)
                s = want[r].sum(0)
                t = e[r].sum(0) + (n + 16) * 2.0 ** -24 * want[r].abs().sum(0) + ref.rounding(s, BF16) * 1.01
                ref.assert_near(db[g], s, t, f"dbias of group {g}")


def test_epilogue_backward_in_place_and_no_rows():
    z, dy = rand(1, 70, 32), rand(2, 70, 32)
    want, _ = tg.epilogue_backward(dy.cuda(), z.cuda(), "gelu")
    for which in range(2):
        zc, dc = z.cuda(), dy.cuda()
        got, _ = tg.epilogue_backward(dc, zc, "gelu", dz=(zc, dc)[which])
        assert torch.equal(got, want)
    dz, db = tg.epilogue_backward(torch.empty(0, 32, dtype=BF16, device="cuda"), torch.empty(0, 32, dtype=BF16, device="cuda"),
                                  "relu")
    assert dz.shape == (0, 32) and (db == 0).all()


# --------------------------------------------------------------------------
# The experts' products
# --------------------------------------------------------------------------
def groups_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


COUNTS = [[3, 0, 17, 1, 0], [0, 0], [64, 130, 5], [1] * 70, [0, 300, 0, 9]]


def run_grouped(counts, N, K, dtype, trans, act, gather, bias=True, preact=True, seed=0, spare=5):
    E, off = len(counts), groups_of(counts)
    used = int(off[-1])
    R = used + spare
    F = N // 2 if act in ref.GATED else N
    b = rand(seed, E, N, K, dtype=dtype, scale=1 / math.sqrt(K))
    bd = b.cuda().transpose(1, 2) if trans else b.transpose(1, 2).contiguous().cuda()
    bs = rand(seed + 1, E, N, dtype=dtype) if bias else None
    if gather:
        S = 29
        a = rand(seed + 2, S, K, dtype=dtype)
        rows = torch.randint(0, S, (R,), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        if used > 3:
            rows[1], rows[2], rows[3] = -1, S, 2 ** 30
        inside = (rows >= 0) & (rows < S)
        ar = torch.where(inside[:, None], a[rows.clamp(0, S - 1).long()], torch.zeros(1, dtype=dtype))
    else:
        a = ar = rand(seed + 2, R, K, dtype=dtype)
        rows = None
    out = torch.full((R, F), 3.0, dtype=dtype, device="cuda")
    z = torch.full((R, N), 5.0, dtype=dtype, device="cuda") if preact else None
    say("grouped", counts[:6], N, K, dtype, trans, act, gather)
    tg.gemm_grouped(a.cuda(), bd, off.cuda(), rows=None if rows is None else rows.cuda(),
                    bias=None if bs is None else bs.cuda(), act=act, preact=z, out=out)
    torch.cuda.synchronize()
    assert (out[used:].cpu() == 3.0).all(), "rows behind the last group were written"
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        yr, ty, zr, tz = ref.epilogue(ar[lo:hi], b[e].t(), None if bs is None else bs[e], act, None, dtype)
        ref.assert_near(out[lo:hi], yr, ty, f"group {e}")
        if preact:
            ref.assert_near(z[lo:hi], zr, tz, f"preact of group {e}")
    if preact:
        assert (z[used:].cpu() == 5.0).all()


@pytest.mark.parametrize("size", [16, 64, 128, 256])
@pytest.mark.parametrize("counts", COUNTS, ids=["few", "none", "many", "ones", "one"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(size, counts, gather, tile):
    tile(size, size)
    run_grouped(counts, 136, 200, BF16, True, "silu", gather, seed=size)
    run_grouped(counts, 48, 72, F16, True, "swiglu", gather, preact=not gather, seed=size + 1)


@pytest.mark.parametrize("size", [64, 128, 256])
def test_grouped_weights_stored_k_by_n(size, tile):
    tile(size, size)
    for counts in COUNTS:
        run_grouped(counts, 264, 136, BF16, False, "none", False, bias=False, preact=False, seed=size)
        run_grouped(counts, 80, 72, BF16, False, "geglu", True, seed=size + 1)


@pytest.mark.parametrize("size", [64, 128, 256])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("act", ["none", "swiglu", "geglu"])
def test_grouped_with_nothing_else(size, gather, trans, act, tile):
    """No bias and no preact: the instances that store straight from the
    accumulators.  Last tiles of up to half a tile's rows and of more, K of one
    slice, of a few and of more than the prefetch looks ahead, N of several
    tiles and a ragged one."""
    tile(size, size)
    N = 520 if act == "none" else 528
    for i, (counts, K) in enumerate([([300, 0, 140, 256, 1, 520], 328), ([64, 129, 383, 5], 72), ([2, 0, 128], 584)]):
        run_grouped(counts, N, K, F16 if i == 1 else BF16, trans, act, gather, bias=False, preact=False, seed=size + i)
        run_grouped(counts[:3], 48, K, BF16 if i == 1 else F16, trans, act, gather, bias=False, preact=False, seed=i)


@pytest.mark.parametrize("size", [16, 64, 128, 256])
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
def test_grouped_with_an_empty_k(size, act, tile):
    """Nothing to sum: the bias through the activation, or zeros, in every row
    of a group and none behind."""
    tile(size, size)
    counts, N = [3, 0, 140, 1], 48
    off, used = groups_of(counts), sum(counts)
    F = N // 2 if act in ref.GATED else N
    bias = rand(1, 4, N)
    for bs in (bias, None):
        for trans in (True, False) if size != 16 else (True,):
            b = torch.empty(4, N, 0, dtype=BF16, device="cuda").transpose(1, 2) if trans else torch.empty(4, 0, N, dtype=BF16, device="cuda")
            out = torch.full((used + 2, F), 3.0, dtype=BF16, device="cuda")
            say("grouped, K = 0", size, act, trans, bs is not None)
            tg.gemm_grouped(torch.empty(used + 2, 0, dtype=BF16, device="cuda"), b, off.cuda(), bias=None if bs is None else bs.cuda(),
                            act=act, out=out)
            torch.cuda.synchronize()
            assert (out[used:] == 3.0).all()
            for e, n in enumerate(counts):
                z = (torch.zeros(1, N) if bs is None else bs[e:e + 1]).double()
                want = ref.layer(z, act)
                tol = ref.layer_error(z, torch.zeros_like(z), act) + ref.rounding(want, BF16) * 1.001
                lo = int(off[e])
                ref.assert_near(out[lo:lo + n], want.expand(n, F), tol.expand(n, F), f"group {e}")


def test_no_rows_at_all():
    """Empty row sets: nothing is written but the gradients' zeros."""
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    rows = torch.empty(0, dtype=torch.int32, device="cuda")
    x, y = (torch.empty(0, n, dtype=BF16, device="cuda") for n in (72, 136))
    w = rand(1, 3, 72, 136).cuda()
    out = torch.full((3, 72, 136), 3.0, dtype=BF16, device="cuda")
    assert not tg.gemm_grouped_tn(x, y, off, out=out).any()
    assert tg.gemm_grouped(x, w, off).shape == (0, 136)
    assert tg.gemm_grouped(x, w, off, rows=rows).shape == (0, 136)
    # Rows of a source that has none read zeros.
    got = tg.gemm_grouped(x, w, torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda"),
                          rows=torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert got.shape == (5, 136) and not got.any()
    assert tg.expert_gather(x, rows).shape == (0, 72)
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert tg.expert_combine(x, none).shape == (0, 72)
    slots = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    res = rand(2, 6, 72).cuda()
    assert torch.equal(tg.expert_combine(x, slots, residual=res), res)
    dh, dw = tg.expert_combine_backward(res, x, slots, torch.ones(6, 2, device="cuda"))
    torch.cuda.synchronize()
    assert dh.shape == (0, 72) and not dw.any()
    z, db = tg.epilogue_backward(y, y, "silu", offsets=off)
    assert z.shape == (0, 136) and db.shape == (3, 136) and not db.any()


def test_grouped_chosen_kernels():
    run_grouped([200, 1, 300, 77], 520, 264, BF16, True, "gelu", False, seed=1)
    run_grouped([20, 1, 33, 0, 17], 520, 264, BF16, True, "gelu", True, seed=2)
    run_grouped([40, 60, 33, 0, 64], 528, 264, F16, True, "swiglu", True, seed=3)


def test_grouped_offsets_that_are_none_touch_nothing_else():
    """Falling, negative and far offsets: what is computed is unspecified, but
    only rows of the output are written."""
    for size in (16, 64):
        ffn.set_tile(size, size)
        try:
            for off in ([0, 40, 20, 64], [-5, 10, 1 << 30, 64], [64, 0, 0, 0], [70, 80, 90, 100]):
                big = torch.full((64 + 16, 48), 3.0, dtype=BF16, device="cuda")
                a, b = rand(1, 64, 72).cuda(), rand(2, 3, 48, 72).cuda()
                say("offsets", off, size)
                tg.gemm_grouped(a, b.transpose(1, 2), torch.tensor(off, dtype=torch.int32, device="cuda"), out=big[8:72])
                torch.cuda.synchronize()
                assert (big[:8] == 3.0).all() and (big[72:] == 3.0).all()
        finally:
            ffn.set_tile()


def test_grouped_weights_in_a_larger_array(tile):
    """A stride between the matrices and between their rows."""
    for size in (16, 128):
        tile(size, size)
        E, N, K, counts = 3, 40, 72, [5, 0, 20]
        big = torch.full((E, N + 3, K + 16), float("nan"), dtype=BF16, device="cuda")
        b = rand(1, E, N, K)
        big[:, 1:N + 1, 8:K + 8] = b.cuda()
        a, off = rand(2, 25, K), groups_of(counts)
        y = tg.gemm_grouped(a.cuda(), big[:, 1:N + 1, 8:K + 8].transpose(1, 2), off.cuda())
        torch.cuda.synchronize()
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if hi > lo:
                yr, ty, _, _ = ref.epilogue(a[lo:hi], b[e].t(), None, "none", None, BF16)
                ref.assert_near(y[lo:hi], yr, ty)


@pytest.mark.parametrize("size", [0, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_tn(size, dtype, tile):
    tile(size, size)
    for counts in COUNTS + [[63, 64, 65, 128, 2]]:
        off = groups_of(counts)
        R = int(off[-1]) + 3
        for P, Q in ((8, 8), (136, 264)):
            x, y = rand(1, R, P, dtype=dtype), rand(2, R, Q, dtype=dtype)
            x[int(off[-1]):] = float("nan")       # rows in no group take no part
            out = torch.full((len(counts), P, Q), 3.0, dtype=dtype, device="cuda")
            say("grouped_tn", counts[:6], P, Q, dtype, size)
            tg.gemm_grouped_tn(x.cuda(), y.cuda(), off.cuda(), out=out)
            torch.cuda.synchronize()
            for e in range(len(counts)):
                lo, hi = int(off[e]), int(off[e + 1])
                xe, ye = x[lo:hi].double().t(), y[lo:hi].double()
                want = xe @ ye
                ref.assert_near(out[e], want, ref.product_error(xe, ye) + ref.rounding(want, dtype) * 1.001,
                                f"group {e}")


# --------------------------------------------------------------------------
# Together, and how they are called
# --------------------------------------------------------------------------
def close_on_the_whole(got, want, dtype, steps, what):
    """A chain of rounded operators: the difference's norm within so many half
    steps of the result's."""
    got, want = got.detach().cpu().double(), want.detach().double()
    assert got.shape == want.shape
    off, norm = float((got - want).norm()), float(want.norm())
    assert off <= steps * ref.EPS[dtype] * norm + 1e-30, f"{what}: {off / norm:.3g} off"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_two_layers_with_their_gradients(dtype, act):
    """A feed-forward block with a residual, forward and backward, against
    automatic differentiation in 64 bits.  Each gradient passes at most six
    roundings (two of them inside a derivative of slope below 1.13)."""
    M, D, H = 150, 72, 136
    N = 2 * H if act in ref.GATED else H
    x, w1, b1 = rand(1, M, D, dtype=dtype), rand(2, N, D, dtype=dtype, scale=0.12), rand(3, N, dtype=dtype)
    w2, b2, dy = rand(4, D, H, dtype=dtype, scale=0.09), rand(5, D, dtype=dtype), rand(6, M, D, dtype=dtype)
    X, W1, B1, W2, B2, DY = (t.cuda() for t in (x, w1, b1, w2, b2, dy))
    z = torch.empty(M, N, dtype=dtype, device="cuda")
    h = tg.gemm_epilogue(X, W1.t(), bias=B1, act=act, preact=z)
    y = tg.gemm_epilogue(h, W2.t(), bias=B2, residual=X)
    _, db2 = tg.epilogue_backward(DY, None, "none")
    dw2 = tg.gemm(DY.t(), h)
    dz, db1 = tg.epilogue_backward(tg.gemm(DY, W2), z, act)
    dw1 = tg.gemm(dz.t(), X)
    dx = tg.gemm_epilogue(dz, W1, residual=DY)
    torch.cuda.synchronize()
    p = [t.double().requires_grad_() for t in (x, w1, b1, w2, b2)]
    yr = ref.layer(p[0] @ p[1].t() + p[2], act) @ p[3].t() + p[4] + p[0]
    yr.backward(dy.double())
    for got, want, what in ((y, yr, "y"), (dx, p[0].grad, "dx"), (dw1, p[1].grad, "dw1"), (db1, p[2].grad, "db1"),
                            (dw2, p[3].grad, "dw2"), (db2, p[4].grad, "db2")):
        close_on_the_whole(got, want, dtype, 6, what)


def expert_layer(x, logits, w1, b1, w2, dy, k, act):
    """Forward and backward of an expert layer with the library's operators."""
    w, ids = tg.route_topk(logits, k)
    offsets, rows, slots = tg.route_plan(ids, logits.shape[1])
    xs = tg.expert_gather(x, rows)
    z = torch.empty(rows.numel(), w1.shape[1], dtype=x.dtype, device=x.device)
    h = tg.gemm_grouped(xs, w1.transpose(1, 2), offsets, bias=b1, act=act, preact=z)
    o = tg.gemm_grouped(h, w2.transpose(1, 2), offsets)
    y = tg.expert_combine(o, slots, w, residual=x)
    do, dw = tg.expert_combine_backward(dy, o, slots, w)
    dw2 = tg.gemm_grouped_tn(do, h, offsets)
    dz, db1 = tg.epilogue_backward(tg.gemm_grouped(do, w2, offsets), z, act, offsets=offsets)
    dw1 = tg.gemm_grouped_tn(dz, xs, offsets)
    dx = tg.expert_combine(tg.gemm_grouped(dz, w1, offsets), slots, residual=dy)
    dl = tg.route_topk_backward(dw, logits, ids)
    fused = tg.gemm_grouped(x, w1.transpose(1, 2), offsets, rows=rows, bias=b1, act=act)
    return {"y": y, "dx": dx, "dw1": dw1, "db1": db1, "dw2": dw2, "dlogits": dl, "h": h, "fused": fused}


def expert_inputs(dtype, T, E, D, H, act, seed=0):
    N = 2 * H if act in ref.GATED else H
    return (rand(seed, T, D, dtype=dtype), rand(seed + 1, T, E, dtype=dtype), rand(seed + 2, E, N, D, dtype=dtype, scale=0.12),
            rand(seed + 3, E, N, dtype=dtype), rand(seed + 4, E, D, H, dtype=dtype, scale=0.09), rand(seed + 5, T, D, dtype=dtype))


@pytest.mark.parametrize("counts,N,K", [([1, 0, 2, 0, 0, 3, 1, 1], 2048, 136), ([2, 1, 1], 4096, 2056), ([1] * 24, 2048, 200),
                                        ([3, 0, 1, 0], 272, 2048)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_grouped_few_rows_by_choice(counts, N, K, act):
    """Numbers of experts hit that take 64 x 64 tiles, and the kernel for few
    rows with four and with eight waves, by the library's own choice."""
    run_grouped(counts, N, K, BF16, True, act, True, seed=len(counts))


@pytest.mark.parametrize("M,N,K", [(16, 16384, 64), (9, 10240, 136), (8, 10240, 136), (5, 8264, 2048), (2, 24, 2048)])
def test_few_rows_by_choice(M, N, K):
    run_epilogue(M, N, K, BF16, "nt", "silu", seed=M)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
@pytest.mark.parametrize("T,E,k", [(120, 5, 2), (3, 40, 3)])
def test_expert_layer_with_its_gradients(dtype, act, T, E, k):
    """Against automatic differentiation in 64 bits over the same choices; at
    most eight roundings to a gradient, the router's through differences of
    numbers up to some times its size."""
    D, H = 72, 136
    ins = expert_inputs(dtype, T, E, D, H, act)
    got = expert_layer(*(t.cuda() for t in ins), k, act)
    torch.cuda.synchronize()
    x, logits, w1, b1, w2 = (t.double().requires_grad_() for t in ins[:5])
    _, ids = ref.topk(ins[1], k)
    s = torch.softmax(logits, 1).gather(1, ids)
    w = s / s.sum(1, keepdim=True)
    y = x + 0
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            y = y + torch.zeros_like(y).index_add(0, torch.tensor([t]), (w[t, j] * (ref.layer(x[t] @ w1[e].t() + b1[e], act) @ w2[e].t()))[None])
    y.backward(ins[5].double())
    for name, want, steps in (("y", y, 8), ("dx", x.grad, 8), ("dw1", w1.grad, 8), ("db1", b1.grad, 8),
                              ("dw2", w2.grad, 8), ("dlogits", logits.grad, 32)):
        close_on_the_whole(got[name], want, dtype, steps, name)
    assert torch.equal(got["fused"], got["h"]), "gathered rows give other results than their copies"


def test_expert_layer_of_a_padded_batch():
    """Tokens whose logits are all masked, tokens with one expert left, an
    expert that nobody may choose, and memory that held NaN before: what has
    no expert keeps its residual and has no gradient."""
    T, E, k, D, H, act, dtype = 90, 6, 3, 72, 136, "swiglu", BF16
    x, logits, w1, b1, w2, dy = expert_inputs(dtype, T, E, D, H, act, seed=7)
    logits[:, 4] = -math.inf
    logits[50:] = -math.inf
    logits[60:] = float("nan")
    logits[10:20, 1:] = -math.inf
    nan = [torch.full((T * k, n), float("nan"), dtype=dtype, device="cuda") for n in (D, D, D, H, H, 2 * H, 2 * H)]
    torch.cuda.synchronize()
    del nan
    got = expert_layer(*(t.cuda() for t in (x, logits, w1, b1, w2, dy)), k, act)
    torch.cuda.synchronize()
    xr, w1r, b1r, w2r = (t.double().requires_grad_() for t in (x, w1, b1, w2))
    lr = torch.where(torch.isfinite(logits.double()), logits.double(), torch.zeros(())).requires_grad_()
    _, ids = ref.topk(logits, k)
    rows = []
    for t in range(T):
        y, chosen = xr[t], [int(e) for e in ids[t] if e >= 0]
        if chosen:
            v = torch.softmax(lr[t, chosen], 0)
            y = y + sum(v[j] * (ref.layer(xr[t] @ w1r[e].t() + b1r[e], act) @ w2r[e].t()) for j, e in enumerate(chosen))
        rows.append(y)
    y = torch.stack(rows)
    y.backward(dy.double())
    for name, want, steps in (("y", y, 8), ("dx", xr.grad, 8), ("dw1", w1r.grad, 8), ("db1", b1r.grad, 8),
                              ("dw2", w2r.grad, 8), ("dlogits", lr.grad, 32)):
        close_on_the_whole(got[name], want, dtype, steps, name)
    assert torch.equal(got["y"][50:].cpu(), x[50:]) and torch.equal(got["dx"][50:].cpu(), dy[50:])
    assert not got["dlogits"][50:].any() and not got["dlogits"][:, 4].any()
    assert not got["dw1"][4].any() and not got["db1"][4].any() and not got["dw2"][4].any()


def test_offsets_past_32_bits():
    """Outputs of more than 4 GiB: their last rows, and the moves between them."""
    M, N, K = 262400, 8200, 64
    x, w = rand(1, M, K), rand(2, 2, N, K, scale=0.1)
    X, W = x.cuda(), w.cuda()
    res, z, out = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(3))
    tail = rand(3, 70, N)
    res[-70:] = tail.cuda()
    assert out.numel() * 2 > 1 << 32
    say("past 32 bits", M, N)
    tg.gemm_epilogue(X, W[0].t(), act="relu", residual=res, preact=z, out=out)
    torch.cuda.synchronize()
    yr, ty, zr, tz = ref.epilogue(x[-70:], w[0].t(), None, "relu", tail, BF16)
    ref.assert_near(out[-70:], yr, ty, "out")
    ref.assert_near(z[-70:], zr, tz, "preact")
    say("gradient")
    dz, _ = tg.epilogue_backward(out, z, "relu", want_dbias=False, dz=res)
    torch.cuda.synchronize()
    assert torch.equal(dz[-70:], out[-70:] * (z[-70:] > 0))
    say("grouped")
    off = torch.tensor([0, M - 70, M], dtype=torch.int32, device="cuda")
    tg.gemm_grouped(X, W.transpose(1, 2), off, act="relu", preact=z, out=out)
    torch.cuda.synchronize()
    yr, ty, zr, tz = ref.epilogue(x[-70:], w[1].t(), None, "relu", None, BF16)
    ref.assert_near(out[-70:], yr, ty, "grouped out")
    ref.assert_near(z[-70:], zr, tz, "grouped preact")
    say("rows")
    back = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    tg.expert_gather(out, back, out=z)
    torch.cuda.synchronize()
    assert torch.equal(z[:70], out[-70:].flip(0)) and torch.equal(z[-70:], out[:70].flip(0))
    tg.expert_combine(z, back[:, None], out=res)
    torch.cuda.synchronize()
    assert torch.equal(res[-70:], out[-70:]) and torch.equal(res[:70], out[:70])
    two = torch.full((M, 1), 2.0, device="cuda")
    dh, dw = tg.expert_combine_backward(out, z, back[:, None], two, dh=res)
    torch.cuda.synchronize()
    assert torch.equal(dh[:70], 2 * out[-70:].flip(0)) and torch.equal(dh[-70:], 2 * out[:70].flip(0))
    want = (out[-70:].double() ** 2).sum(1)   # sums of up to 8200 binary32 products, all positive
    assert bool(((dw[-70:, 0].double() - want).abs() <= 8200 * 2.0 ** -24 * want + 1e-30).all())


def test_the_same_inputs_give_the_same_bits():
    ins = [t.cuda() for t in expert_inputs(BF16, 300, 9, 136, 264, "swiglu", seed=3)]
    first = expert_layer(*ins, 2, "swiglu")
    first = {k: v.clone() for k, v in first.items()}
    for _ in range(3):
        again = expert_layer(*ins, 2, "swiglu")
        for name, v in first.items():
            assert torch.equal(again[name], v), name


def test_graph_replays_match_eager():
    """An expert layer with its gradients captured once and replayed over
    changed inputs, with eager work between the replays."""
    ins = [t.cuda() for t in expert_inputs(BF16, 64, 6, 72, 136, "gelu", seed=1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        expert_layer(*ins, 2, "gelu")
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = expert_layer(*ins, 2, "gelu")
    for i in range(4):
        for t, n in zip(ins, expert_inputs(BF16, 64, 6, 72, 136, "gelu", seed=20 + i)):
            t.copy_(n)
        want = {k: v.clone() for k, v in expert_layer(*ins, 2, "gelu").items()}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, v in want.items():
            assert torch.equal(got[name], v), (i, name)


def test_other_streams_and_threads():
    """Two threads at once, each on a stream of its own, with different tiles."""
    a, b = rand(1, 96, 264).cuda(), rand(2, 136, 264).cuda()
    want = {}
    for size in (16, 128):
        ffn.set_tile(size, size)
        want[size] = tg.gemm_epilogue(a, b.t(), act="silu")
    ffn.set_tile()
    torch.cuda.synchronize()
    errors = []

    def work(size):
        try:
            s = torch.cuda.Stream()
            ffn.set_tile(size, size)
            for _ in range(20):
                y = tg.gemm_epilogue(a, b.t(), act="silu", stream=s)
                dz, db = tg.epilogue_backward(y, y, "silu", stream=s)
                s.synchronize()
                assert torch.equal(y, want[size])
            with pytest.raises(tg.TgemmError):
                tg.gemm_epilogue(a, b.t(), out=a[:, :136])
        except BaseException as e:   # noqa: BLE001 - handed to the test
            errors.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in (16, 128)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors


def test_the_binding_refuses():
    a, b = torch.zeros(8, 16, dtype=BF16, device="cuda"), torch.zeros(16, 24, dtype=BF16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        tg.gemm_epilogue(a, b[:8])
    with pytest.raises(TypeError):
        tg.gemm_epilogue(a, b.half())
    with pytest.raises(ValueError):
        tg.gemm_epilogue(a, b, act="tanh")
    with pytest.raises(ValueError):
        tg.gemm_epilogue(a, b, bias=b[0, :8])
    with pytest.raises(ValueError):
        tg.gemm_epilogue(a, b, residual=a)
    with pytest.raises(ValueError):
        tg.gemm_epilogue(a, b.cpu())
    with pytest.raises(TypeError):
        tg.gemm_epilogue(a, b, out=torch.zeros(8, 24, device="cuda"))
    with pytest.raises(ValueError):
        tg.gemm_epilogue(a, b, out=torch.zeros(8, 48, dtype=BF16, device="cuda")[:, ::2])
    with pytest.raises(TypeError):
        tg.gemm_grouped(a, b[None], off[:2].long())
    with pytest.raises(ValueError):
        tg.gemm_grouped(a, b[None], off)
    with pytest.raises(ValueError):
        tg.epilogue_backward(a, None, "relu")
    with pytest.raises(ValueError):
        tg.route_topk(a.float(), 2, score="max")
    with pytest.raises(tg.TgemmError):
        tg.route_topk(a.float(), 17)


def test_flags_that_are_no_truth_values_are_refused():
    """An array of several values has no truth value: a TypeError, not a result
    beside an error."""
    x = rand(1, 8, 16).cuda()
    several = torch.tensor([True, False])
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for call, name in ((lambda: tg.epilogue_backward(x, x, "relu", want_dbias=several), "want_dbias"),
                       (lambda: tg.route_topk(x, 2, renormalize=several), "renormalize"),
                       (lambda: tg.route_topk_backward(torch.zeros(8, 2, device="cuda"), x, ids, renormalize=several), "renormalize")):
        with pytest.raises(TypeError, match=name + " must be true or false"):
            call()
    dz, db = tg.epilogue_backward(x, x, "relu", want_dbias=torch.tensor(False))
    assert db is None and dz.shape == x.shape
