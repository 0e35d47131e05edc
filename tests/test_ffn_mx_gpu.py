"""MXFP4 on the GPU: quantisation and back bit for bit against the definition;
the products with an epilogue, dense and by expert, against their 64-bit form:
every kernel, activation and type, sizes that end anywhere, scale rows in any
alignment, NaN scales, strides, empty groups, gradients, graphs, streams."""
import math

import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn
import _ffn_more_ref as more
import _ffn_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
#: The kernels, by the tile that forces each; 0 is the library's own choice.
TILES = [0, 16, 64, 128, 256]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()


@pytest.fixture
def tile():
    def force(size, K):
        """256 x 256 tiles take whole slices of 256 elements; other K go by the library's own choice."""
        size = 0 if size == 256 and K % 256 else size
        ffn.set_tile(size, size)

    yield force
    ffn.set_tile()


def rand(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def rand_mx(seed, rows, K, spread=3):
    """Random elements and scales around 1 (K / 32 a row)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(127 - spread, 128 + spread, (rows, K // 32), generator=g, dtype=torch.uint8)
    return q, s


def say(*what):
    print("[gpu]", *what, flush=True)


# --------------------------------------------------------------------------
# Quantisation
# --------------------------------------------------------------------------
def same_bits(got, want, what):
    for g, w, n in zip(got, want, ("elements", "scales")):
        assert torch.equal(g.cpu(), w), (what, n, int((g.cpu() != w).sum()))


def check_quant(x, columns=True):
    xg = x.cuda()
    rows = x.shape[1] % 32 == 0
    if rows:
        same_bits(tg.quantize_mxfp4(xg), more.quantize(x), "rows")
    if columns:
        t = more.quantize(x.t())
        same_bits(tg.quantize_mxfp4(xg, rows=False, columns=True), t, "columns")
        if rows:
            both = tg.quantize_mxfp4(xg, columns=True)
            same_bits(both[:2], more.quantize(x), "rows of both")
            same_bits(both[2:], t, "columns of both")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,N", [(1, 32), (1, 2080), (3, 64), (31, 96), (32, 32), (33, 128), (129, 160), (200, 2048),
                                 (65, 72), (7, 8), (130, 40)])
def test_quantize(M, N, dtype):
    say("quantize", M, N, dtype)
    check_quant(rand(M + N, M, N, dtype=dtype, scale=3.0) * torch.exp(2 * rand(1, M, 1, dtype=F32)).to(dtype))


def test_quantize_every_rounding():
    """Values at, just below and just above each border between elements, both
    signs, at scales over binary32's range; the block's largest is 6."""
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    base = []
    for v in borders:
        base += [v, v * (1 - 2.0 ** -23), v * (1 + 2.0 ** -22)]
    base += [0.0, 1e-30, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 5.9, 6.0, 0.2]
    base = torch.tensor(base, dtype=F32)
    assert base.numel() == 32
    rows = []
    for e in (-120, -60, -3, 0, 1, 40, 120):
        for sign in (1, -1):
            rows.append(sign * base * 2.0 ** e)
    check_quant(torch.stack(rows))
    b = torch.tensor(borders + [0.0, 6.0, 4.0, 3.0, 2.0, 1.0, 0.5, 1.5, 0.125], dtype=F32)
    x = torch.cat((b, -b)).to(BF16)
    check_quant(torch.stack([x * 2.0 ** e for e in (-30, 0, 5)]).to(BF16))
    check_quant(torch.stack([x.float() * 2.0 ** e for e in (-3, 0, 5)]).to(F16))


def test_quantize_every_scale():
    """The largest value on either side of 6 times each power of two, subnormal ones, the largest numbers, zeros."""
    tops = []
    for e in range(-127, 126):
        six = 6.0 * 2.0 ** e
        tops += [six, six * (1 + 2.0 ** -23), six * (1 - 2.0 ** -24)]
    tops += [0.0, -0.0, 2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 3.4028234663852886e38]
    x = torch.zeros(len(tops), 32, dtype=F32)
    x[:, 5] = torch.tensor(tops, dtype=torch.float64).to(F32)
    x[:, 9] = -x[:, 5] / 3
    x[:, 11] = -0.0
    check_quant(x)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quantize_every_16_bit_value(dtype):
    """Each as the largest of its block, with parts of it beside; in rows and columns."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    v = torch.zeros(65536, 32, dtype=dtype)
    v[:, 0] = x
    for i, part in enumerate((0.04, 0.05, 0.1, 0.13, 0.2, 0.21, 0.3, 0.42, 0.5, 0.6, 0.84, 0.99)):
        v[:, 2 + i] = (x.float() * (part if i % 2 else -part)).to(dtype)
    same_bits(tg.quantize_mxfp4(v.cuda()), more.quantize(v), "rows")
    u = v[::7].t().contiguous()
    same_bits(tg.quantize_mxfp4(u[:, :9344].contiguous().cuda(), rows=False, columns=True), more.quantize(u[:, :9344].t()), "columns")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_not_finite(dtype):
    x = rand(3, 70, 96, dtype=dtype)
    x[0, 3], x[1, 40], x[2, 95], x[40, 0] = math.inf, -math.inf, math.nan, math.nan
    check_quant(x)
    q, s = tg.quantize_mxfp4(x.cuda())
    v = tg.dequantize_mxfp4(q, s, dtype=F32).cpu()
    assert torch.isnan(v[0, :32]).all() and torch.isfinite(v[0, 32:]).all() and torch.isnan(v[2, 64:]).all()


def test_quantize_strides_and_places():
    buf = rand(1, 50, 160).cuda()
    x = buf[:, 16:16 + 96]
    want = tg.quantize_mxfp4(x.contiguous(), columns=True)
    q = torch.full((50, 80), 17, dtype=torch.uint8, device="cuda")
    qt = torch.full((96, 64), 17, dtype=torch.uint8, device="cuda")
    got = tg.quantize_mxfp4(x, columns=True, q=q[:, 16:64], qt=qt[:, 16:48])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (q[:, :16] == 17).all() and (q[:, 64:] == 17).all() and (qt[:, :16] == 17).all() and (qt[:, 48:] == 17).all()
    assert all(torch.equal(a, b) for a, b in zip(tg.quantize_mxfp4(x), want[:2]))
    v = torch.full((50, 128), 3.0, dtype=BF16, device="cuda")
    tg.dequantize_mxfp4(got[0], got[1], out=v[:, 8:104])
    assert torch.equal(v[:, 8:104], tg.dequantize_mxfp4(*want[:2])) and (v[:, :8] == 3).all() and (v[:, 104:] == 3).all()


def test_quantize_nothing():
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    q, s, qt, st = tg.quantize_mxfp4(x, columns=True)
    assert q.shape == (0, 32) and s.shape == (0, 2) and qt.shape == (64, 0) and st.shape == (64, 0)
    assert tg.dequantize_mxfp4(q, s).shape == (0, 64)


def test_quantize_a_fresh_row_of_every_width():
    for N in range(32, 32 * 70, 32 * 7):
        check_quant(rand(N, 3, N), columns=False)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_dequantize(dtype):
    """Every element at every scale."""
    q = torch.arange(256, dtype=torch.uint8).view(1, 256).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 16)
    got = tg.dequantize_mxfp4(q.cuda(), s.cuda(), dtype=dtype).cpu()
    want = more.values(q, s).to(dtype)
    assert got.dtype == dtype
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok]) and torch.equal(torch.signbit(got[ok]), torch.signbit(want[ok]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_past_the_largest(dtype):
    """Exactly what is below 2^128; from there on infinities, to which finite numbers
    can be quantised."""
    q = torch.tensor([[0x10, 0x32, 0x54, 0x76] * 4] * 3, dtype=torch.uint8, device="cuda")
    s = torch.tensor([[252], [253], [254]], dtype=torch.uint8, device="cuda")
    got = tg.dequantize_mxfp4(q, s, dtype=dtype).cpu().double()
    want = more.values(q.cpu(), s.cpu())
    assert torch.equal(torch.isinf(got), want >= 2.0 ** 128)
    assert torch.isinf(got).sum(1).tolist() == [0, 8, 16] and torch.equal(got[want < 2.0 ** 128], want[want < 2.0 ** 128])
    x = torch.zeros(2, 32, dtype=dtype, device="cuda")
    x[0, 3], x[1, 3] = 1.75 * 2.0 ** 127, -1.7421875 * 2.0 ** 127      # (the bfloat16 before)
    back = tg.dequantize_mxfp4(*tg.quantize_mxfp4(x), dtype=dtype)
    assert back[0, 3] == math.inf and back[1, 3] == -1.5 * 2.0 ** 127


# --------------------------------------------------------------------------
# Products with an epilogue
# --------------------------------------------------------------------------
def run_epilogue(M, N, K, dtype=BF16, act="none", bias=True, residual=True, preact=True, seed=0):
    say("mx epilogue", M, N, K, dtype, act, bias, residual, preact)
    F = N // 2 if act in ref.GATED else N
    a, sa = rand_mx(seed, M, K)
    b, sb = rand_mx(seed + 1, N, K)
    sb = (sb.int() - int(math.log2(max(K, 1)) / 2) - 2).to(torch.uint8)     # sums of about unit size
    bs = rand(seed + 2, N, dtype=dtype) if bias else None
    rs = rand(seed + 3, M, F, dtype=dtype) if residual else None
    z = torch.full((M, N), 7.0, dtype=dtype, device="cuda") if preact else None
    y = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), bias=None if bs is None else bs.cuda(), act=act,
                               residual=None if rs is None else rs.cuda(), preact=z, dtype=dtype)
    torch.cuda.synchronize()
    yr, ty, zr, tz = more.product(a, sa, b, sb, bs, act, rs, dtype)
    assert y.dtype == dtype
    if dtype == F16:
        # Half a step past the largest binary16 (65520 and on) rounds to infinity.
        over = torch.isinf(y.cpu()) & (yr.abs() + ty >= 65520) & (y.cpu().sign() == yr.sign())
        y = torch.where(over, yr, y.cpu().double())
    ref.assert_near(y, yr, ty, "out")
    if preact:
        ref.assert_near(z, zr, tz, "preact")


SIZES = [(1, 8, 32), (1, 264, 1024), (3, 40, 96), (16, 16, 512), (17, 136, 544), (33, 48, 160), (64, 72, 2080),
         (130, 200, 1056), (300, 264, 288), (257, 520, 4128), (70, 72, 256), (300, 264, 512), (130, 520, 1280), (513, 8, 4096)]


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_products(M, N, K, dtype, size, tile):
    tile(size, K)
    run_epilogue(M, N, K, dtype, "none", seed=M + N + K)
    run_epilogue(M, N, K, dtype, ACTS[(M + K // 32) % 5], bias=M % 2 == 0, residual=M % 3 == 0, preact=N % 16 == 8, seed=N)
    run_epilogue(M, N, K, dtype, bias=False, residual=False, preact=False, seed=K)


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("act", ref.GATED)
@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (5, 80, 224), (31, 48, 1056), (50, 1040, 320), (300, 528, 544), (67, 272, 96),
                                   (300, 528, 256), (70, 16, 768), (260, 272, 1536)])
def test_products_gated(act, M, N, K, size, tile):
    tile(size, K)
    run_epilogue(M, N, K, BF16, act, residual=M % 2 == 1, seed=M)
    run_epilogue(M, N, K, F16, act, bias=False, residual=False, preact=False, seed=M + 9)


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("act", ACTS)
def test_activations(act, size, tile):
    tile(size, 256)
    run_epilogue(256, 256, 512, BF16, act, seed=4)
    run_epilogue(72, 136, 256, F16, act, seed=5)


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("K", [32 * i for i in range(1, 20)] + [1024 + 32 * i for i in range(1, 18, 3)] + [2048, 2560, 4096])
def test_every_tail_of_k(K, size, tile):
    tile(size, K)
    run_epilogue(70, 72, K, BF16, "none", residual=False, preact=False, seed=K)


@pytest.mark.parametrize("M,N,K,act", [(17, 72, 8192, "gelu"), (100, 256, 8224, "silu"), (300, 136, 9312, "relu"),
                                       (64, 1024, 16384, "none"), (130, 272, 8288, "swiglu"), (40, 1040, 7200, "geglu")])
def test_split_k(M, N, K, act):
    assert ffn.lib().tgemm_mxfp4_workspace_bytes(M, N, K) > 0
    run_epilogue(M, N, K, BF16, act, seed=M)
    run_epilogue(M, N, K, F16, act, bias=False, residual=False, preact=False, seed=M + 9)


def test_split_k_workspaces():
    """The sums stay within the bytes asked for; with a byte less K is not
    split; a replayed graph has the same bits."""
    M, N, K = 100, 256, 8224
    a, sa = (t.cuda() for t in rand_mx(0, M, K))
    b, sb = (t.cuda() for t in rand_mx(1, N, K))
    need = ffn.lib().tgemm_mxfp4_workspace_bytes(M, N, K)
    guard = torch.full((need + 256,), 165, dtype=torch.uint8, device="cuda")
    want = tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="silu", workspace=guard[:need])
    assert (guard[need:] == 165).all() and (guard[:need] != 165).any()
    guard.fill_(165)
    less = tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="silu", workspace=guard[:need - 16])
    assert (guard == 165).all()
    _, tol, _, _ = more.product(a.cpu(), sa.cpu(), b.cpu(), sb.cpu(), None, "silu", None, BF16)
    ref.assert_near(less, want.cpu().double(), 2 * tol)
    assert torch.equal(tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="silu"), want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="silu", out=out, workspace=guard[:need])
    for _ in range(3):
        out.zero_()
        guard.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_split_k_nan_scales():
    M, N, K = 70, 72, 8288
    a, sa = rand_mx(1, M, K)
    b, sb = rand_mx(2, N, K)
    clean = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
    sa[1, 0], sa[33, -1], sb[5, 0], sb[64, -1] = 255, 255, 255, 255
    got = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
    hit = torch.zeros(M, N, dtype=torch.bool)
    hit[[1, 33]] = True
    hit[:, [5, 64]] = True
    assert torch.isnan(got.cpu()[hit]).all() and torch.equal(got.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("size", TILES)
def test_products_of_whole_numbers_are_exact(size, tile):
    """Sums of small whole numbers fit binary32 and the output: every bit counts."""
    for M, N, K in [(5, 40, 96), (130, 136, 544), (260, 264, 256), (513, 520, 1024)]:
        tile(size, K)
        g = torch.Generator().manual_seed(K)
        codes = torch.tensor([0, 2, 4, 10, 12, 0, 0, 0])          # 0, 1, 2, -1, -2
        pick = lambda r: codes[torch.randint(0, 8, (r, K), generator=g)].to(torch.uint8)
        pack = lambda c: c[:, 0::2] | (c[:, 1::2] << 4)
        a, b = pack(pick(M)), pack(pick(N))
        sa, sb = (torch.randint(126, 129, (r, K // 32), generator=g, dtype=torch.uint8) for r in (M, N))
        want = more.values(a, sa) @ more.values(b, sb).t()
        got = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
        assert torch.equal(got.cpu(), want.to(BF16))


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("K", [32, 96, 544, 1056, 256, 512, 1280])
def test_nan_scales_stay_in_their_rows(K, size, tile):
    """A NaN block makes its row (or column) NaN, and no other: not the row
    before it either, whose blocks end right before its own in memory."""
    tile(size, K)
    M, N = 70, 72
    a, sa = rand_mx(1, M, K)
    b, sb = rand_mx(2, N, K)
    clean = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
    sa[1, 0], sa[33, -1], sb[5, 0], sb[64, -1] = 255, 255, 255, 255
    got = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
    hit = torch.zeros(M, N, dtype=torch.bool)
    hit[[1, 33]] = True
    hit[:, [5, 64]] = True
    assert torch.isnan(got.cpu()[hit]).all()
    assert torch.equal(got.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_scales_from_any_address(shift, size, tile):
    tile(0 if size == 256 else size, 0)       # (256 x 256 tiles take scales from a dword on)
    for K in (256, 512, 96, 4096):
        M, N = 40, 72
        a, sa = rand_mx(1, M, K)
        b, sb = rand_mx(2, N, K)
        want = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())

        def moved(s, by):
            buf = torch.full((s.numel() + 16,), 255, dtype=torch.uint8, device="cuda")
            v = buf[by:by + s.numel()].view(s.shape)
            v.copy_(s)
            return v

        got = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), moved(sa, shift), moved(sb, 4 - shift))
        assert torch.equal(got, want)


@pytest.mark.parametrize("size", TILES)
def test_strides_and_places(size, tile):
    for M, N, K in [(9, 72, 96), (150, 136, 544), (260, 264, 512)]:
        tile(size, K)
        a, sa = (t.cuda() for t in rand_mx(1, M, K))
        b, sb = (t.cuda() for t in rand_mx(2, N, K))
        rs = rand(3, M, N).cuda()
        want = tg.gemm_mxfp4_epilogue(a, b, sa, sb, residual=rs, act="silu")
        wide = lambda t, pad: torch.nn.functional.pad(t, (pad, pad), value=0x77)[:, pad:-pad]
        c = torch.full((M, N + 32), 5.0, dtype=BF16, device="cuda")
        c[:, 8:8 + N] = rs
        view = c[:, 8:8 + N]
        tg.gemm_mxfp4_epilogue(wide(a, 16), wide(b, 32), sa, sb, residual=view, act="silu", out=view)
        assert torch.equal(view, want) and (c[:, :8] == 5).all() and (c[:, 8 + N:] == 5).all()


def test_nothing_to_multiply():
    e = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    bias = rand(0, 16).cuda()
    y = tg.gemm_mxfp4_epilogue(e(3, 0), e(16, 0), e(3, 0), e(16, 0), bias=bias)
    assert torch.equal(y, bias.expand(3, 16))
    assert tg.gemm_mxfp4_epilogue(e(0, 32), e(16, 32), e(0, 2), e(16, 2)).shape == (0, 16)
    assert tg.gemm_mxfp4_epilogue(e(3, 32), e(0, 32), e(3, 2), e(0, 2)).shape == (3, 0)


@pytest.mark.parametrize("size", [0, 16, 64, 128])
@pytest.mark.parametrize("M", [1, 70, 300, 20000])
def test_an_empty_k(M, size, tile):
    """Each kernel's loop over no K at all, null operands: the epilogue of zeros."""
    tile(size, 0)
    N, E = 40, 3
    e = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    bias, rs = rand(0, N).cuda(), rand(1, M, N).cuda()
    z = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    y = tg.gemm_mxfp4_epilogue(e(M, 0), e(N, 0), e(M, 0), e(N, 0), bias=bias, act="relu", residual=rs, preact=z)
    assert torch.equal(z, bias.expand(M, N))
    assert torch.equal(y, (bias.float().relu() + rs.float()).to(BF16))
    assert (tg.gemm_mxfp4_epilogue(e(M, 0), e(N, 0), e(M, 0), e(N, 0)) == 0).all()
    off = torch.tensor([0, M // 2, M // 2, M], dtype=torch.int32, device="cuda")
    src = torch.arange(M, dtype=torch.int32, device="cuda").flip(0)
    for rows in (None, src):
        z.fill_(7.0)
        b3 = rand(2, E, N).cuda()
        tg.gemm_mxfp4_grouped(e(M, 0), e(E, N, 0), e(M, 0), e(E, N, 0), off, rows=rows, bias=b3, out=z)
        assert torch.equal(z[:M // 2], b3[0].expand(M // 2, N)) and torch.equal(z[M // 2:], b3[2].expand(M - M // 2, N))


def test_the_plain_product_agrees():
    """gemm_mxfp4_nt on the same operands: sums in another order, each rounded once."""
    for M, N, K in [(300, 264, 1024), (256, 512, 96)]:
        a, sa = rand_mx(1, M, K)
        b, sb = rand_mx(2, N, K)
        old = tg.gemm_mxfp4_nt(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
        _, tol, _, _ = more.product(a, sa, b, sb, None, "none", None, BF16)
        got = tg.gemm_mxfp4_epilogue(a.cuda(), b.cuda(), sa.cuda(), sb.cuda())
        ref.assert_near(got, old.cpu().double(), 2 * tol)


@pytest.mark.parametrize("M", [1, 33, 96, 129, 256, 257, 600])
def test_the_plain_product_takes_quantised_columns(M):
    """Whatever M is: the rows of quantised columns lie apart where 16 bytes a block of
    32 are no whole cache lines.  Either operand, both, and an output given."""
    x, y = rand(M, M, 96), rand(M + 1, M, 72)
    _, _, xt, sx = tg.quantize_mxfp4(x.cuda(), columns=True)
    yt, sy = tg.quantize_mxfp4(y.cuda(), rows=False, columns=True)
    assert xt.is_contiguous() == (-(-M // 32) * 16 % 128 == 0)
    a, b = more.values(*more.quantize(x.t())), more.values(*more.quantize(y.t()))
    want, tol, _, _ = ref.epilogue(a, b.t(), None, "none", None, BF16)
    out = torch.empty(96, 72, dtype=BF16, device="cuda")
    for p, q in ((xt, yt), (xt.contiguous(), yt), (xt, yt.contiguous())):
        ref.assert_near(tg.gemm_mxfp4_nt(p, q, sx, sy), want, tol)
        got = tg.gemm_mxfp4_nt(p, q, sx, sy, out=out, stream=torch.cuda.current_stream())
        assert got.data_ptr() == out.data_ptr()
        ref.assert_near(out, want, tol)
    with pytest.raises(ValueError, match="row-major"):
        tg.gemm_mxfp4_nt(xt.t().contiguous().t(), yt, sx, sy)
    with pytest.raises(ValueError, match="contiguous"):
        tg.gemm_mxfp4_nt(xt, yt, sx, sy, out=torch.empty(72, 96, dtype=BF16, device="cuda").t())


# --------------------------------------------------------------------------
# By expert
# --------------------------------------------------------------------------
def run_grouped(sizes, N, K, dtype=BF16, act="none", gather=True, bias=True, preact=True, seed=0, tail=3):
    """Groups of these sizes, `tail` rows behind the last left alone."""
    E = len(sizes)
    F = N // 2 if act in ref.GATED else N
    R = sum(sizes) + tail
    S = max(R // 2, 1) if gather else R
    say("mx grouped", sizes, N, K, dtype, act, gather, bias, preact)
    a, sa = rand_mx(seed, S, K)
    b, sb = rand_mx(seed + 1, E * N, K)
    sb = (sb.int() - int(math.log2(K) / 2) - 2).to(torch.uint8)
    bs = rand(seed + 2, E, N, dtype=dtype) if bias else None
    g = torch.Generator().manual_seed(seed + 3)
    rows = torch.randint(0, S, (R,), generator=g, dtype=torch.int32) if gather else None
    if gather and R > 4:
        rows[1], rows[3] = -1, S          # outside: zeros
    off = torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32)
    z = torch.full((R, N), 7.0, dtype=dtype, device="cuda") if preact else None
    out = torch.full((R, F), 9.0, dtype=dtype, device="cuda")
    got = tg.gemm_mxfp4_grouped(a.cuda(), b.cuda().view(E, N, -1), sa.cuda(), sb.cuda().view(E, N, -1), off.cuda(),
                                rows=None if rows is None else rows.cuda(), bias=None if bs is None else bs.cuda(), act=act,
                                preact=z, out=out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    av = more.values(a, sa)
    bv = more.values(b, sb).view(E, N, K)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        if gather:
            idx = rows[lo:hi].long()
            ok = (idx >= 0) & (idx < S)
            x = torch.where(ok[:, None], av[idx.clamp(0, S - 1)], torch.zeros(1, dtype=torch.float64))
        else:
            x = av[lo:hi]
        yr, ty, zr, tz = ref.epilogue(x, bv[e].t(), None if bs is None else bs[e], act, None, dtype)
        ref.assert_near(out[lo:hi], yr, ty, f"group {e}")
        if preact:
            ref.assert_near(z[lo:hi], zr, tz, f"preact of group {e}")
    end = sum(sizes)
    assert (out[end:] == 9).all() and (z is None or (z[end:] == 7).all())


GROUPS = [[1], [0, 3, 0], [1, 2, 0, 5, 17], [40, 0, 130, 7], [300, 1, 64], [129, 257, 0, 0, 16]]


@pytest.mark.parametrize("size", TILES)
@pytest.mark.parametrize("sizes", GROUPS, ids=str)
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(sizes, gather, size, tile):
    for i, (N, K, dtype, act, rest) in enumerate([
            (72, 96, BF16, "gelu", {}), (136, 544, F16, "none", dict(bias=False, preact=False)),
            (272, 512, BF16, "swiglu", dict(bias=False, preact=False)), (80, 1056, F16, "geglu", {}),
            (40, 256, BF16, "relu", dict(preact=False, tail=0)), (520, 768, F16, "none", dict(bias=False, preact=False)),
            (528, 256, F16, "geglu", {})]):
        tile(size, K)
        run_grouped(sizes, N, K, dtype, act, gather, seed=len(sizes) + i, **rest)


def test_grouped_many_small_groups():
    run_grouped([i % 4 for i in range(150)], 48, 160, BF16, "silu", seed=8)


@pytest.mark.parametrize("size", TILES)
def test_grouped_offsets_are_clamped(size, tile):
    """Offsets that leave the rows: nothing outside is touched."""
    N, K, R = 72, 256, 20
    tile(size, K)
    a, sa = (t.cuda() for t in rand_mx(0, R, K))
    b, sb = (t.cuda().view(2, N, -1) for t in rand_mx(1, 2 * N, K))
    whole = torch.full((R + 8, N), 9.0, dtype=BF16, device="cuda")
    off = torch.tensor([-5, 12, 1000], dtype=torch.int32, device="cuda")
    tg.gemm_mxfp4_grouped(a, b, sa, sb, off, out=whole[4:4 + R])
    want = tg.gemm_mxfp4_grouped(a, b, sa, sb, torch.tensor([0, 12, R], dtype=torch.int32, device="cuda"))
    assert torch.equal(whole[4:4 + R], want) and (whole[:4] == 9).all() and (whole[4 + R:] == 9).all()


def test_grouped_weights_apart():
    """Experts' weights and scales with room between them."""
    E, N, K, R = 3, 40, 96, 12
    a, sa = (t.cuda() for t in rand_mx(0, R, K))
    b, sb = (t.cuda().view(E, N, -1) for t in rand_mx(1, E * N, K))
    off = torch.tensor([0, 4, 5, 12], dtype=torch.int32, device="cuda")
    want = tg.gemm_mxfp4_grouped(a, b, sa, sb, off)
    bb = torch.full((E, N + 3, K // 2 + 16), 255, dtype=torch.uint8, device="cuda")
    bb[:, :N, :K // 2] = b
    ss = torch.full((E, N + 1, K // 32), 255, dtype=torch.uint8, device="cuda")
    ss[:, :N] = sb
    assert torch.equal(tg.gemm_mxfp4_grouped(a, bb[:, :N, :K // 2], sa, ss[:, :N], off), want)


@pytest.mark.parametrize("size", TILES)
def test_grouped_one_weight_for_all(size, tile):
    """One weight for every group (strides of 0), and every row gathered from the same
    token.  Products are multiples of 2^-6 of at most 48 x 12: sums of 256 fit 24 bits,
    and every kernel gives the same."""
    E, N, K, R = 70, 48, 256, 300
    a, sa = (t.cuda() for t in rand_mx(0, 3, K))
    b, sb = (t.cuda() for t in rand_mx(1, N, K, spread=1))
    tile(size, K)
    want = tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="relu")
    off = torch.linspace(0, R, E + 1).int().cuda()
    for e in (E, 7):                        # (more groups than a wave has lanes, and fewer)
        ends = off[:e + 1].clone()
        rows = torch.full((R,), 2, dtype=torch.int32, device="cuda")
        out = torch.full((R, N), 9.0, dtype=BF16, device="cuda")
        tg.gemm_mxfp4_grouped(a, b.expand(e, N, K // 2), sa, sb.expand(e, N, K // 32), ends, rows=rows, act="relu", out=out)
        n = int(ends[-1])
        assert torch.equal(out[:n], want[2:3].expand(n, N)) and (out[n:] == 9).all()


@pytest.mark.parametrize("size", [0, 16])
@pytest.mark.parametrize("K", [96, 160, 1024])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_few_rows_of_many_weight_rows(K, dtype, size, tile):
    """The kernel for few rows where a wave takes two blocks of weight rows (more than
    32 a compute unit, by all groups that have rows), the last ones incomplete."""
    tile(size, K)
    run_epilogue(3, 8264, K, dtype, "silu", seed=K)
    run_epilogue(16, 8232, K, dtype, bias=False, residual=False, preact=False, seed=K + 1)
    sizes = [(7 * i) % 5 for i in range(40)]
    run_grouped(sizes, 264, K, dtype, "gelu", True, seed=K + 2)
    run_grouped(sizes, 248, K, dtype, "none", False, bias=False, preact=False, seed=K + 3)


# --------------------------------------------------------------------------
# Together
# --------------------------------------------------------------------------
def test_a_linear_layers_gradients():
    """Forward and both gradients on quantised operands, odd rows; each is the
    product of the quantised matrices, which the definition gives exactly."""
    M, N, K = 77, 96, 160
    x, w, dy = rand(0, M, K), rand(1, N, K, scale=0.1), rand(2, M, N)
    xa = tg.quantize_mxfp4(x.cuda(), columns=True)
    wa = tg.quantize_mxfp4(w.cuda(), columns=True)
    da = tg.quantize_mxfp4(dy.cuda(), columns=True)
    mul = lambda p, i, q, j: tg.gemm_mxfp4_epilogue(p[i], q[j], p[i + 1], q[j + 1])
    y, dx, dw = mul(xa, 0, wa, 0), mul(da, 0, wa, 2), mul(da, 2, xa, 2)
    for got, p, q in ((y, x, w), (dx, dy, w.t()), (dw, dy.t(), x.t())):
        a, b = more.values(*more.quantize(p)), more.values(*more.quantize(q))
        want, tol, _, _ = ref.epilogue(a, b.t(), None, "none", None, BF16)
        ref.assert_near(got, want, tol)


def test_a_layer_of_experts_behind_its_norm():
    """Norm, routing, quantisation, both products of the experts, combination:
    each step against the definition on what the step before it gave."""
    T, E, k, D, H = 37, 6, 2, 96, 64
    x = rand(0, T, D)
    g, b = rand(1, D, dtype=F32), rand(2, D, dtype=F32)
    logits = rand(3, T, E)
    w1, w2 = rand(4, E, 2 * H, D, scale=0.1), rand(5, E, D, H, scale=0.1)
    q = lambda w: tuple(t.view(E, w.shape[1], -1) for t in tg.quantize_mxfp4(w.cuda().view(-1, w.shape[2])))
    (b1, s1), (b2, s2) = q(w1), q(w2)
    n = tg.layer_norm(x.cuda(), g.cuda(), b.cuda())
    wts, ids = tg.route_topk(logits.cuda(), k)
    off, rows, slots = tg.route_plan(ids, E)
    a, sa = tg.quantize_mxfp4(n)
    h = tg.gemm_mxfp4_grouped(a, b1, sa, s1, off, rows=rows, act="swiglu")
    a2, sa2 = tg.quantize_mxfp4(h)
    y = tg.gemm_mxfp4_grouped(a2, b2, sa2, s2, off)
    out = tg.expert_combine(y, slots, wts, residual=x.cuda())
    nr, nt = more.layer_norm(x, g, b, 1e-5, BF16)[:2]
    ref.assert_near(n, nr, nt, "norm")
    same_bits((a, sa), more.quantize(n.cpu()), "rows")
    av, hv = more.values(*more.quantize(n.cpu())), more.values(*more.quantize(h.cpu()))
    o, r = off.cpu(), rows.cpu().long()
    for e in range(E):
        lo, hi = int(o[e]), int(o[e + 1])
        if lo == hi:
            continue
        yr, ty, _, _ = ref.epilogue(av[r[lo:hi]], more.values(*more.quantize(w1[e])).t(), None, "swiglu", None, BF16)
        ref.assert_near(h[lo:hi], yr, ty, "first product")
        yr, ty, _, _ = ref.epilogue(hv[lo:hi], more.values(*more.quantize(w2[e])).t(), None, "none", None, BF16)
        ref.assert_near(y[lo:hi], yr, ty, "second product")
    want = x.double() + (y.cpu().double()[slots.cpu().long()] * wts.cpu().double()[:, :, None]).sum(1)
    tol = ref.rounding(want, BF16) * 1.001 + 1e-6 * (1 + want.abs())
    ref.assert_near(out, want, tol, "layer")


def test_same_bits_in_graphs_and_on_streams():
    M, N, K = 70, 264, 544
    x = rand(0, M, K).cuda()
    b, sb = (t.cuda() for t in rand_mx(1, N, K))
    bias = rand(2, N).cuda()

    def step(out=None):
        a, sa = tg.quantize_mxfp4(x)
        return tg.gemm_mxfp4_epilogue(a, b, sa, sb, bias=bias, act="silu", out=out)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert torch.equal(want, other)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(out)
    for i in range(4):
        x.copy_(rand(10 + i, M, K))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


def test_chosen_kernels():
    """Sizes that take each kernel by the library's own choice: few rows, one and
    two 64 x 64 tiles a CU, 128 x 128, 256 x 256."""
    for M, N, K, act in [(16, 4096, 512, "silu"), (64, 4096, 1088, "gelu"), (600, 3000, 320, "none"), (1030, 2056, 288, "relu"),
                         (4100, 4104, 256, "none"), (1500, 4112, 96, "swiglu")]:
        run_epilogue(M, N, K, BF16, act, seed=M)
        run_epilogue(M, N, K, F16, act, bias=True, residual=False, preact=False, seed=M)


def test_calls_from_threads_at_once():
    import threading

    M, N, K = 200, 264, 1056
    a, sa = (t.cuda() for t in rand_mx(0, M, K))
    b, sb = (t.cuda() for t in rand_mx(1, N, K))
    x = rand(2, M, 512).cuda()
    want, q = tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="silu"), tg.quantize_mxfp4(x, columns=True)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                y, p = tg.gemm_mxfp4_epilogue(a, b, sa, sb, act="silu"), tg.quantize_mxfp4(x, columns=True)
                s.synchronize()
                if not torch.equal(y, want) or not all(torch.equal(i, j) for i, j in zip(p, q)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_padded_batch():
    """Rows behind the last group (ids -1 in the routing) have no part in anything."""
    T, E, k, D, H = 40, 5, 2, 64, 96
    x = rand(0, T, D)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    ids[30:] = -1
    w = rand(2, E, H, D, scale=0.1)
    b, sb = (t.view(E, H, -1) for t in tg.quantize_mxfp4(w.cuda().view(-1, D)))
    off, rows, slots = tg.route_plan(ids.cuda(), E)
    a, sa = tg.quantize_mxfp4(x.cuda())
    out = torch.full((T * k, H), 9.0, dtype=BF16, device="cuda")
    tg.gemm_mxfp4_grouped(a, b, sa, sb, off, rows=rows, out=out)
    n = int(off[-1])
    assert n == 60 and (out[n:] == 9).all() and (out[:n] != 9).any()
    y = tg.expert_combine(out, slots)
    assert (y[30:] == 0).all()


def test_types_follow_what_is_given():
    a, sa = (t.cuda() for t in rand_mx(0, 4, 64))
    b, sb = (t.cuda() for t in rand_mx(1, 16, 64))
    half = torch.zeros(16, dtype=F16, device="cuda")
    assert tg.gemm_mxfp4_epilogue(a, b, sa, sb).dtype == BF16
    assert tg.gemm_mxfp4_epilogue(a, b, sa, sb, bias=half).dtype == F16
    assert tg.gemm_mxfp4_epilogue(a, b, sa, sb, out=torch.empty(4, 16, dtype=F16, device="cuda")).dtype == F16
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    assert tg.gemm_mxfp4_grouped(a, b[None], sa, sb[None], off, bias=half[None]).dtype == F16
    with pytest.raises(TypeError, match="bfloat16 or torch.float16"):
        tg.gemm_mxfp4_epilogue(a, b, sa, sb, dtype=F32)
    with pytest.raises(TypeError, match="bias must be torch.bfloat16"):
        tg.gemm_mxfp4_epilogue(a, b, sa, sb, bias=half, dtype=BF16)
