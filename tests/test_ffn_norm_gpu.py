"""The layer norm and its gradients on the GPU against the plain 64-bit forms
and against differences: types, widths of every kernel, strides, in place,
rows far from zero, graphs, streams."""
import math

import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn
import _ffn_more_ref as more
import _ffn_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
#: Widths around every change of kernel.
WIDTHS = [8, 64, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 5000, 8192, 8200, 16384, 16392, 20000]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()


def rand(seed, *shape, dtype=BF16, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def say(*what):
    print("[gpu]", *what, flush=True)


def run(M, N, dtype=BF16, wdtype=None, weight=True, bias=True, residual=True, eps=1e-5, seed=0, scale=1.0, shift=0.0):
    wdtype = wdtype or dtype
    say("norm", M, N, dtype, wdtype, weight, bias, residual)
    x = rand(seed, M, N, dtype=dtype, scale=scale, shift=shift)
    w = rand(seed + 1, N, dtype=wdtype, scale=0.3, shift=1.0) if weight else None
    b = rand(seed + 2, N, dtype=wdtype, scale=0.2) if bias else None
    dy = rand(seed + 3, M, N, dtype=dtype)
    rs = rand(seed + 4, M, N, dtype=dtype) if residual else None
    g = lambda t: None if t is None else t.cuda()
    mean, rstd = (torch.full((M,), 7.0, device="cuda") for _ in range(2))
    xg = g(x)
    y = tg.layer_norm(xg, g(w), g(b), eps=eps, mean=mean, rstd=rstd)
    dx, dw, db = tg.layer_norm_backward(g(dy), xg, g(w), mean, rstd, residual=g(rs))
    torch.cuda.synchronize()
    yr, ty, mu, r, tmu, tr, _, _ = more.layer_norm(x, w, b, eps, dtype)
    ref.assert_near(y, yr, ty, "y")
    ref.assert_near(mean, mu, tmu, "mean")
    ref.assert_near(rstd, r, tr, "rstd")
    back = more.layer_norm_backward(dy, x, w, eps, rs, dtype, wdtype if weight else dtype)
    for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
        ref.assert_near(got, *back[name], name)
    assert y.dtype == dx.dtype == dtype
    assert dw.dtype == db.dtype == (wdtype if weight else dtype)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_widths(N, dtype):
    run(5, N, dtype, F32 if N % 3 == 0 else None, residual=N % 16 == 0, seed=N)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 63, 64, 65, 257, 1100])
@pytest.mark.parametrize("N", [72, 520, 2056])
def test_rows(M, N):
    run(M, N, BF16 if M % 2 else F16, F32 if M % 3 else None, residual=M % 2 == 0, seed=M)


@pytest.mark.parametrize("M,N", [(9001, 8), (4500, 504), (5001, 520), (2301, 1024), (2900, 1032), (1301, 2056), (700, 4104),
                                 (530, 8192)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rows_in_several_turns(M, N, dtype):
    """More rows than all workgroups of the gradients take at once: 4096 of up to 512
    values, 2048 of up to 1024, 1024 of up to 2048, 512 of up to 4096, 256 of up to 8192."""
    run(M, N, dtype, F32 if N % 3 == 0 else None, residual=N % 16 == 0, seed=M)


@pytest.mark.parametrize("M,N", [((1 << 22) + 5003, 8), ((1 << 20) + 5003, 520), ((1 << 20) + 3, 1032), (600001, 2056), (270001, 8192),
                                 (70001, 8200)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_column_sums_of_many_rows_are_exact(M, N, dtype):
    """Whole numbers, whose sums binary32 holds in any order: no row is left out or
    counted twice, where the workgroups' sums go to the workspace more than once (from
    513 turns on) and where they do not.  And dx of rows of later turns."""
    say("column sums", M, N, dtype)
    g = torch.Generator(device="cuda").manual_seed(N)
    x, dy = (torch.empty(M, N, dtype=dtype, device="cuda").random_(-2, 3, generator=g) for _ in range(2))
    mean, rstd, w = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    dx, dw, db = tg.layer_norm_backward(dy, x, w, mean, rstd)
    want = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    step = max((1 << 26) // N, 1)
    for lo in range(0, M, step):
        d, v = dy[lo:lo + step].float(), x[lo:lo + step].float()
        want += torch.stack(((d * v).sum(0, dtype=torch.float64), d.sum(0, dtype=torch.float64)))
    assert want.abs().max() < 2 ** 24
    assert torch.equal(dw.double(), want[0]) and torch.equal(db.double(), want[1])
    for lo in (M // 2, M - 40):
        part = slice(lo, lo + 40)
        few = tg.layer_norm_backward(dy[part].clone(), x[part].clone(), w, mean[:40], rstd[:40], want_dweight=False)[0]
        assert torch.equal(dx[part], few)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(weight, bias):
    run(37, 264, BF16, F32 if weight else None, weight=weight, bias=bias, residual=False)
    if not weight and bias:
        x, b = rand(0, 4, 64), rand(1, 64, dtype=F32)
        ref.assert_near(tg.layer_norm(x.cuda(), bias=b.cuda()), *more.layer_norm(x, None, b, 1e-5, BF16)[:2], "y")


@pytest.mark.parametrize("N", [256, 3000, 17000])
def test_rows_far_from_zero_keep_their_digits(N):
    """The variance of rows whose mean is a thousand times their spread."""
    run(9, N, F32, shift=1000.0, seed=3)
    run(9, N, BF16, scale=100.0, shift=-3000.0, seed=4)


def test_small_and_large_rows():
    run(6, 1024, F32, scale=1e-18, seed=5)
    run(6, 1024, F32, scale=1e15, seed=6)
    run(6, 1024, F32, eps=0.0, seed=7)


def test_rows_of_equal_values():
    x = torch.full((3, 64), 2.5, dtype=BF16, device="cuda")
    b = rand(0, 64).cuda()
    assert torch.equal(tg.layer_norm(x, None, b), b.expand(3, 64))


def test_a_row_with_nan_or_infinity_is_its_own_affair():
    x = rand(0, 6, 2056, dtype=BF16)
    clean = tg.layer_norm(x.cuda())
    x[1, 7], x[3, 2000] = math.nan, math.inf
    y = tg.layer_norm(x.cuda())
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    for r in (0, 2, 4, 5):
        assert torch.equal(y[r], clean[r])


def test_strides_and_places():
    """Rows apart, outputs inside larger arrays left as they were around them, in place."""
    M, N, ld = 11, 264, 296
    for dtype in (BF16, F32):
        buf = rand(1, M, ld, dtype=dtype).cuda()
        x = buf[:, 8:8 + N]
        w, b = rand(2, N, dtype=dtype).cuda(), rand(3, N, dtype=dtype).cuda()
        dy, rs = rand(4, M, N, dtype=dtype).cuda(), rand(5, M, N, dtype=dtype).cuda()
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        want = tg.layer_norm(x.contiguous(), w, b, mean=mean, rstd=rstd)
        out = torch.full((M, ld), 3.0, dtype=dtype, device="cuda")
        tg.layer_norm(x, w, b, out=out[:, 16:16 + N])
        assert torch.equal(out[:, 16:16 + N], want)
        assert (out[:, :16] == 3).all() and (out[:, 16 + N:] == 3).all()
        grads = tg.layer_norm_backward(dy, x.contiguous(), w, mean, rstd, residual=rs)
        for into in ("dout", "x", "residual"):
            t = {"dout": dy.clone(), "x": x.contiguous().clone(), "residual": rs.clone()}
            got = tg.layer_norm_backward(t["dout"], t["x"], w, mean, rstd, residual=t["residual"], dx=t[into])
            assert got[0] is not None and all(torch.equal(p, q) for p, q in zip(got, grads)), into
        big = torch.full((M, ld), 3.0, dtype=dtype, device="cuda")
        got = tg.layer_norm_backward(dy, x, w, mean, rstd, residual=rs, dx=big[:, 8:8 + N])
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
        assert (big[:, :8] == 3).all() and (big[:, 8 + N:] == 3).all()
        same = x.contiguous().clone()
        assert torch.equal(tg.layer_norm(same, w, b, out=same), want)


def test_gradients_without_the_weights():
    x, dy = rand(0, 70, 520), rand(1, 70, 520)
    mean, rstd = torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    w = rand(2, 520).cuda()
    tg.layer_norm(x.cuda(), w, mean=mean, rstd=rstd)
    dx, dw, db = tg.layer_norm_backward(dy.cuda(), x.cuda(), w, mean, rstd)
    only, a, b = tg.layer_norm_backward(dy.cuda(), x.cuda(), w, mean, rstd, want_dweight=False)
    assert a is None and b is None and torch.equal(only, dx)


def test_no_rows():
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    m = torch.zeros(0, device="cuda")
    assert tg.layer_norm(x).shape == (0, 64)
    dx, dw, db = tg.layer_norm_backward(x, x, None, m, m)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("N", [64, 2056])
def test_gradients_against_differences(N):
    """Along random directions in binary32: the difference quotient of the
    64-bit form with step t is off by t^2 / 6 of a third derivative, and the
    gradient by its tolerance's sum."""
    M, t = 7, 1e-4
    x, w, b, dy = (rand(i, *s, dtype=F32) for i, s in enumerate([(M, N), (N,), (N,), (M, N)]))
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    tg.layer_norm(x.cuda(), w.cuda(), b.cuda(), mean=mean, rstd=rstd)
    got = tg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    f = lambda x, w, b: float((more.layer_norm(x, w, b, 1e-5, F32)[0] * dy.double()).sum())
    back = more.layer_norm_backward(dy, x, w, 1e-5, None, F32, F32)
    for i, (name, var) in enumerate((("dx", x), ("dweight", w), ("dbias", b))):
        v = rand(20 + i, *var.shape, dtype=torch.float64)
        args = [a.double() for a in (x, w, b)]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + t * v, args[i] - t * v
        diff = (f(*up) - f(*down)) / (2 * t)
        along = float((got[i].cpu().double() * v).sum())
        # Third derivatives of a unit-scale norm along v are of the order of the sum of |v dx|.
        room = float((back[name][1] * v.abs()).sum()) + 100 * t * t * float((back[name][0] * v).abs().sum())
        assert abs(diff - along) <= room, (name, diff, along, room)


def test_same_bits_in_graphs_streams_and_with_given_workspaces():
    M, N = 300, 2056
    x, dy, w, b = (t.cuda() for t in (rand(0, M, N), rand(1, M, N), rand(2, N), rand(3, N)))
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    need = ffn.lib().tgemm_layer_norm_backward_workspace_bytes(M, N)
    guard = torch.full((need + 256,), 165, dtype=torch.uint8, device="cuda")
    y = tg.layer_norm(x, w, b, mean=mean, rstd=rstd)
    want = tg.layer_norm_backward(dy, x, w, mean, rstd, workspace=guard[:need])
    assert (guard[need:] == 165).all()
    with pytest.raises(tg.TgemmError) as e:
        tg.layer_norm_backward(dy, x, w, mean, rstd, workspace=guard[:need - 16])
    assert e.value.code == tg.EINVAL
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tg.layer_norm_backward(dy, x, w, mean, rstd, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    outs = [torch.empty_like(t) for t in (y, *want)]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tg.layer_norm(x, w, b, mean=mean, rstd=rstd, out=outs[0])
        tg.layer_norm_backward(dy, x, w, mean, rstd, dx=outs[1], dweight=outs[2], dbias=outs[3], workspace=ws)
    for i in range(4):
        for t in outs:
            t.zero_()
        x.copy_(rand(40 + i, M, N))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        m2, r2 = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        again = [tg.layer_norm(x, w, b, mean=m2, rstd=r2)]
        again += list(tg.layer_norm_backward(dy, x, w, m2, r2))
        assert all(torch.equal(p, q) for p, q in zip(outs, again))


def test_outputs_are_ordinary_tensors():
    """New outputs take part in autograd, belong to inference mode inside it, and
    torch's deterministic mode changes no result."""
    x, w, b = (t.cuda() for t in (rand(0, 9, 264), rand(1, 264), rand(2, 264)))
    y = tg.layer_norm(x, w, b)
    assert not y.requires_grad and not y.is_inference()
    z = y.clone().requires_grad_()
    (z * y).sum().backward()
    assert torch.equal(z.grad, y)
    y2 = tg.layer_norm(x, w, b).requires_grad_()
    (y2 * 2).sum().backward()
    assert (y2.grad == 2).all()
    with torch.inference_mode():
        v = tg.layer_norm(x, w, b)
        assert v.is_inference() and torch.equal(v, y)
        v.add_(1)
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        again = tg.layer_norm(x, w, b)
    finally:
        torch.use_deterministic_algorithms(before)
    assert torch.equal(again, y)


def test_new_outputs_are_seen_by_dispatch_modes_and_profilers():
    """As torch.empty's are: by the operators of both kinds, and the results are the same."""
    from torch.profiler import ProfilerActivity, profile
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(func.overloadpacket.__name__)
            return func(*args, **(kwargs or {}))

    x, w = rand(0, 9, 264).cuda(), rand(1, 264, 264).cuda()
    for call in (lambda: tg.layer_norm(x), lambda: tg.gemm_epilogue(x, w, act="silu")):
        want = call()
        with Seen() as seen:
            got = call()
        assert seen.names == ["empty"] and torch.equal(got, want)
        with profile(activities=[ProfilerActivity.CPU], acc_events=True) as p:
            got = call()
        assert any(e.name == "aten::empty" for e in p.events()) and torch.equal(got, want)
