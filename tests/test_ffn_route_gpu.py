"""Routing to experts on the GPU: the choice, its gradient, the plan and the
moves of rows, against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import dense_tiled_gemm_bf16_amd as tg
from dense_tiled_gemm_bf16_amd import ffn
import _ffn_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    tg.init()
    ffn.lib()


def rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def say(*what):
    print("[gpu]", *what, flush=True)


# Of a weight: the exponential, the sum of up to 1024 terms in a tree, the
# division, the scale: within 32 half steps.
WEIGHT = 32 * 2.0 ** -24


def check_topk(logits, k, **how):
    say("topk", tuple(logits.shape), logits.dtype, k, {a: (v if not isinstance(v, torch.Tensor) else "bias") for a, v in how.items()})
    dev = dict(how)
    if dev.get("bias") is not None:
        dev["bias"] = dev["bias"].cuda()
    w, ids = tg.route_topk(logits.cuda(), k, **dev)
    torch.cuda.synchronize()
    wr, ir = ref.topk(logits, k, how.get("score", "softmax"), how.get("bias"), how.get("groups", 1),
                      how.get("groups_used", 1), how.get("renormalize", True), how.get("scale", 1.0))
    assert w.dtype == F32 and ids.dtype == torch.int32
    other = int((ids.cpu().long() != ir).any(1).sum())
    assert other == 0, f"other experts are chosen in {other} rows"
    ref.assert_near(w, wr, WEIGHT * wr.abs() + 2.0 ** -126, "weights")
    return w, ids


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 3), (7, 8, 2), (33, 64, 6), (40, 97, 8), (17, 128, 16),
                                   (19, 256, 8), (9, 300, 4), (5, 512, 20), (4, 1000, 64), (3, 1024, 1)])
def test_choice(dtype, score, T, E, k):
    x = rand(T + E, T, E, dtype=dtype)
    bias = rand(1, E, scale=0.1)
    for renorm in (True, False):
        check_topk(x, k, score=score, renormalize=renorm, scale=2.5 if renorm else 1.0)
        check_topk(x, k, score=score, bias=bias, renormalize=renorm)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,used,k", [(16, 4, 2, 3), (24, 8, 3, 4), (256, 8, 4, 8), (60, 12, 5, 9), (64, 64, 7, 5),
                                             (16, 16, 4, 4), (320, 10, 2, 12), (1024, 64, 3, 16), (96, 2, 1, 48),
                                             (100, 20, 20, 30)])
def test_choice_by_groups(dtype, score, E, groups, used, k):
    x = rand(E, 21, E, dtype=dtype)
    check_topk(x, k, score=score, groups=groups, groups_used=used, bias=rand(2, E, scale=0.2))
    check_topk(x, k, score=score, groups=groups, groups_used=used, renormalize=False)


def test_ties_go_to_the_lowest_expert():
    x = torch.zeros(6, 40)
    x[1] = 1.5
    x[2, ::3] = 2.0
    x[3, 39] = x[3, 0] = 1.0
    x[4] = torch.finfo(F32).min
    x[5, :20] = -0.0
    for score in ("softmax", "sigmoid"):
        check_topk(x, 7, score=score)
        check_topk(x, 7, score=score, bias=torch.zeros(40))
        check_topk(x, 7, score=score, groups=4, groups_used=2)


def test_masked_logits():
    nan, inf = float("nan"), float("inf")
    x = rand(1, 12, 48)
    x[0] = -inf
    x[1] = nan
    x[2, 1:] = -inf
    x[3, :40] = nan
    x[4, ::2] = -inf
    x[5] = torch.finfo(F32).min
    x[6, 7] = inf
    x[7, 7] = x[7, 9] = inf
    x[8, 3:] = torch.finfo(F32).min
    x[9] = -200.0                      # every sigmoid underflows
    x[10, :] = 100.0
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_topk(x, 10, score=score, renormalize=renorm)
            if score == "sigmoid":
                continue
            check_topk(x[:9], 10, score=score, renormalize=renorm, groups=6, groups_used=3)
            check_topk(x[:9], 10, score=score, renormalize=renorm, bias=rand(3, 48, scale=0.1))
    check_topk(x[:9], 10, score="sigmoid", groups=6, groups_used=3, bias=rand(3, 48, scale=0.1))
    bias = torch.zeros(48)
    bias[5], bias[6] = -inf, nan
    check_topk(rand(2, 9, 48), 46, bias=bias)
    check_topk(rand(2, 9, 48), 48, bias=bias, score="sigmoid")


# Shifts of neighbouring rows: a softmax does not know a row's shift, so its
# choice has to stand beside any other row.
SHIFTS = torch.tensor([0.0, -6.0, -8.0, 5.0, -10.0, 0.0, -12.0, -20.0, 3.0, -200.0])


def check_shifted(x, k, **how):
    w, ids = check_topk(x, k, **how)
    assert bool(((ids >= 0) & (ids < x.shape[1])).all())
    return w, ids


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("E,groups,used,ks", [(48, 1, 1, (1, 6, 20)), (96, 1, 1, (4, 17)), (97, 1, 1, (8,)), (100, 1, 1, (8, 30)),
                                              (127, 1, 1, (3,)), (160, 1, 1, (6,)), (250, 1, 1, (16, 17)), (300, 1, 1, (4,)),
                                              (385, 1, 1, (8,)), (1000, 1, 1, (8,)), (48, 3, 2, (4,)), (96, 6, 3, (6,)),
                                              (100, 20, 5, (8,)), (250, 10, 4, (8,)), (300, 60, 7, (9,)), (320, 64, 5, (8,)),
                                              (576, 64, 64, (8,)), (1000, 8, 3, (8,))])
def test_rows_of_different_scale_with_a_bias(dtype, E, groups, used, ks):
    """Numbers of experts that leave lanes over, between rows whose logits lie
    far above or below, in the last row, and in a row by itself."""
    x = (rand(E, 30, E) + SHIFTS.repeat(3)[:, None]).to(dtype)
    bias = rand(4, E, scale=0.1)
    for k in ks:
        for renorm in (True, False):
            check_shifted(x, k, bias=bias, groups=groups, groups_used=used, renormalize=renorm)
        check_shifted(x, k, bias=torch.zeros(E), groups=groups, groups_used=used)
        check_shifted(x[4:5], k, bias=bias, groups=groups, groups_used=used)
        check_shifted(x, k, score="sigmoid", bias=bias, groups=groups, groups_used=used)
        check_shifted(x, k, groups=groups, groups_used=used, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,used", [(48, 1, 1), (97, 1, 1), (300, 1, 1), (100, 20, 5), (320, 64, 5)])
def test_a_biased_choice_beside_finite_padding(score, E, groups, used):
    """Columns of a larger array whose other columns hold large numbers, and
    rows that are all masked between rows that are not."""
    x = rand(E, 21, E) + SHIFTS.repeat(3)[:21, None]
    x[3], x[11], x[20] = -math.inf, float("nan"), -math.inf
    bias = rand(4, E, scale=0.1)
    how = dict(score=score, bias=bias, groups=groups, groups_used=used)
    wr, ir = ref.topk(x, 6, score, bias, groups, used)
    for pad in (60.0, 3e38, math.inf):
        big = torch.full((21, E + 64), pad, device="cuda")
        big[:, 8:8 + E] = x.cuda()
        say("padding", score, E, groups, pad)
        w, ids = tg.route_topk(big[:, 8:8 + E], 6, **{**how, "bias": bias.cuda()})
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu().long(), ir)
        ref.assert_near(w, wr, WEIGHT * wr.abs() + 2.0 ** -126, "weights")
        check_topk(x, 6, **how)


def test_rows_of_a_larger_array():
    big = torch.full((9, 60), float("nan"), device="cuda")
    x = rand(1, 9, 41)
    big[:, 3:44] = x.cuda()
    w, ids = tg.route_topk(big[:, 3:44], 5)
    wr, ir = ref.topk(x, 5)
    assert torch.equal(ids.cpu().long(), ir)
    ref.assert_near(w, wr, WEIGHT * wr)
    dbig = torch.full((9, 60), 9.0, device="cuda")
    d = tg.route_topk_backward(rand(2, 9, 5).cuda(), big[:, 3:44], ids, dlogits=dbig[:, 3:44])
    assert torch.equal(d, tg.route_topk_backward(rand(2, 9, 5).cuda(), x.cuda(), ids))
    assert (dbig[:, :3] == 9).all() and (dbig[:, 44:] == 9).all()


def test_close_keys_are_ordered_as_in_64_bits():
    """Logits a step apart under a bias that nearly cancels the difference of
    their scores: 32-bit keys would not tell them apart."""
    E, T = 64, 200
    g = torch.Generator().manual_seed(3)
    base = torch.rand(T, 1, generator=g) * 2
    x = (base + torch.arange(E) * 2.0 ** -20).float()
    s = torch.sigmoid(x.double())
    bias = -(s - s.mean(1, keepdim=True)).mean(0).float()
    for score in ("sigmoid", "softmax"):
        check_topk(x, 8, score=score, bias=bias)
        check_topk(x, 8, score=score, bias=bias, groups=8, groups_used=3)


def test_many_tokens():
    x = rand(1, 20011, 72, dtype=BF16)
    w, ids = tg.route_topk(x.cuda(), 4)
    order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(ids.cpu().long(), order)
    assert float((w.sum(1) - 1).abs().max()) < 1e-6


@pytest.mark.parametrize("E,groups", [(64, 4), (48, 8), (480, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_sums_nearly_tie(E, groups, score):
    """Two groups whose scores agree to some 2^-24 at the cut, in both orders:
    the sums in 64 bits decide."""
    T, per = 60, E // groups
    x = rand(1, T, E) - 6.0
    f = torch.exp if score == "softmax" else torch.sigmoid
    inverse = torch.log if score == "softmax" else torch.logit
    a = rand(2, T, 2).double() * 0.3
    b = a[:, 0] - 0.2
    rest = inverse(f(a[:, 0]) + f(a[:, 1]) - f(b))
    for t in range(T):
        first, second = (0, 2) if t % 2 else (2, 0)
        x[t, first * per:first * per + 2] = a[t].float()
        x[t, second * per + 1], x[t, second * per + 3] = float(b[t]), float(rest[t])
    check_topk(x, 2, score=score, groups=groups, groups_used=1)


def test_logits_past_32_bits():
    T, E, k = (1 << 24) + 21, 65, 3
    tail = rand(1, 40, E)
    x = torch.zeros(T, E, dtype=F32, device="cuda")
    x[-40:] = tail.cuda()
    assert x.numel() * 4 > 1 << 32
    say("past 32 bits", T, E)
    w, ids = tg.route_topk(x, k)
    torch.cuda.synchronize()
    wr, ir = ref.topk(tail, k)
    assert torch.equal(ids[-40:].cpu().long(), ir)
    assert float((w[-40:].cpu().double() - wr).abs().max()) < 1e-6
    assert torch.equal(ids[:5].cpu().long(), torch.arange(k).expand(5, k))
    g = torch.zeros(T, k, device="cuda")
    g[-40:] = rand(2, 40, k).cuda()
    d = tg.route_topk_backward(g, x, ids)
    torch.cuda.synchronize()
    t = tail.double().requires_grad_()
    weights_of(t, ir, "softmax", True, 1.0).backward(g[-40:].cpu().double())
    assert float((d[-40:].cpu().double() - t.grad).abs().max()) < 1e-6
    assert not d[:1000].any()


# --------------------------------------------------------------------------
# The gradient
# --------------------------------------------------------------------------
def weights_of(x, ids, score, renorm, scale):
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    sel = s.gather(1, ids)
    return (sel / sel.sum(1, keepdim=True) if renorm else sel) * scale


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_against_differences(score, renorm):
    x = rand(1, 3, 7).double().requires_grad_()
    ids = torch.tensor([[0, 3], [6, 2], [1, 5]])
    g = rand(2, 3, 2).double()
    weights_of(x, ids, score, renorm, 1.5).backward(g)
    h = 1e-6
    for i in range(3):
        for j in range(7):
            d = torch.zeros(3, 7, dtype=torch.float64)
            d[i, j] = h
            num = ((weights_of(x.detach() + d, ids, score, renorm, 1.5)
                    - weights_of(x.detach() - d, ids, score, renorm, 1.5)) * g).sum() / (2 * h)
            assert abs(num - x.grad[i, j]) < 1e-8


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 3), (33, 64, 6), (40, 97, 8), (21, 256, 16), (9, 300, 4), (4, 1000, 64)])
def test_gradient(dtype, score, renorm, T, E, k):
    x, dw = rand(T + E, T, E, dtype=dtype), rand(5, T, k)
    _, ids = tg.route_topk(x.cuda(), k, score=score, renormalize=renorm, scale=2.5)
    say("topk grad", dtype, score, renorm, T, E, k)
    dx = tg.route_topk_backward(dw.cuda(), x.cuda(), ids, score=score, renormalize=renorm, scale=2.5)
    torch.cuda.synchronize()
    p = x.double().requires_grad_()
    at = ids.cpu().long()
    weights_of(p, at, score, renorm, 2.5).backward(dw.double())
    assert dx.dtype == dtype
    # Each term is within WEIGHT of itself; they are added with their signs:
    # the sum of magnitudes bounds both (w_j (|g_j| + sum w |g|)).
    w = weights_of(x.double(), at, score, renorm, 1.0)
    mag = torch.zeros(T, E, dtype=torch.float64)
    total = (w * dw.double().abs() * 2.5).sum(1, keepdim=True)
    if score == "softmax" and not renorm:
        mag += torch.softmax(x.double(), 1) * total
    mag.scatter_add_(1, at, w * (dw.double().abs() * 2.5 + total))
    # (Where the derivative is 0 the reference's own 64-bit terms cancel to
    # within some 2^-53 of their size, not to 0.)
    own = 2.0 ** -48 * total
    ref.assert_near(dx, p.grad, 4 * WEIGHT * mag + own + ref.rounding(p.grad, dtype) * 1.01, "dlogits")


def test_gradient_of_masked_and_missing_choices():
    nan, inf = float("nan"), float("inf")
    x = rand(1, 4, 20)
    x[0] = -inf
    x[1, 3:] = -inf
    x[2, ::2] = nan
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            w, ids = tg.route_topk(x.cuda(), 6, score=score, renormalize=renorm)
            g = rand(2, 4, 6).cuda()
            dx = tg.route_topk_backward(g, x.cuda(), ids, score=score, renormalize=renorm).cpu()
            assert torch.isfinite(dx).all()
            assert (dx[0] == 0).all() and (dx[1, 3:] == 0).all() and (dx[2, ::2] == 0).all()
            # Row 1: as a row of three experts.
            y = x[1:2, :3].contiguous().cuda()
            _, i3 = tg.route_topk(y, 3, score=score, renormalize=renorm)
            want = tg.route_topk_backward(g[1:2, :3].contiguous(), y, i3, score=score, renormalize=renorm)
            ref.assert_near(dx[1:2, :3], want.cpu().double(), 64 * 2.0 ** -24 * torch.ones(1, 3).double() * 8)
    # Ids outside the experts have no gradient.
    ids = torch.tensor([[-1, 20, 2 ** 30, -7]], dtype=torch.int32, device="cuda")
    dx = tg.route_topk_backward(torch.ones(1, 4, device="cuda"), rand(3, 1, 20).cuda(), ids, renormalize=False)
    assert (dx == 0).all()


def test_renormalised_weights_of_scores_too_small():
    """A bias or groups that leave only experts whose scores are far below
    1e-20: a softmax's weights are the softmax over the chosen logits all the
    same, a sigmoid's their sigmoids over their sum + 1e-20.  The gradients go
    by the same formulas."""
    k, E = 4, 96
    x = rand(1, 6, E)
    x[:, 0] = torch.tensor([60.0, 100.0, 200.0, 0.0, 500.0, 80.0])
    bias = torch.zeros(E)
    bias[0] = -math.inf
    w, ids = check_topk(x, k, bias=bias)
    at = ids.cpu().long()
    assert bool((at > 0).all())
    # (p: 5 operations a term on numbers up to 1, and a sum of four.)
    want = torch.softmax(x.double().gather(1, at), 1)
    ref.assert_near(w, want, WEIGHT * want, "softmax")
    dw = rand(2, 6, k)
    p = x.double().requires_grad_()
    torch.softmax(p.gather(1, at), 1).backward(dw.double())
    mag = torch.zeros(6, E, dtype=torch.float64)
    mag.scatter_(1, at, want * (dw.double().abs() + (want * dw.double().abs()).sum(1, keepdim=True)))
    dx = tg.route_topk_backward(dw.cuda(), x.cuda(), ids)
    ref.assert_near(dx, p.grad, 4 * WEIGHT * mag + 2.0 ** -126, "its gradient")

    low = x[:, 1:] * 0.5 - 46.0                    # sigmoids of some 1e-20
    w, ids = check_topk(low, k, score="sigmoid")
    at = ids.cpu().long()
    s = torch.exp(low.double()).gather(1, at)      # (1 + s is 1 here, to 1e-19)
    want = s / (s.sum(1, keepdim=True) + 1e-20)
    assert bool((want.sum(1) < 0.99).any())
    ref.assert_near(w, want, WEIGHT * want, "sigmoid")
    p = low.double().requires_grad_()
    e = torch.exp(p).gather(1, at)
    (e / (e.sum(1, keepdim=True) + 1e-20)).backward(dw.double())
    mag = torch.zeros(6, E - 1, dtype=torch.float64)
    mag.scatter_(1, at, want * (dw.double().abs() + (want * dw.double().abs()).sum(1, keepdim=True)))
    dx = tg.route_topk_backward(dw.cuda(), low.cuda(), ids, score="sigmoid")
    ref.assert_near(dx, p.grad, 4 * WEIGHT * mag + 2.0 ** -126, "its gradient")


def test_gradient_in_place():
    x, dw = rand(1, 50, 64).cuda(), rand(2, 50, 4).cuda()
    _, ids = tg.route_topk(x, 4, renormalize=False)
    want = tg.route_topk_backward(dw, x, ids, renormalize=False)
    got = tg.route_topk_backward(dw, x, ids, renormalize=False, dlogits=x)
    assert torch.equal(got, want)


# --------------------------------------------------------------------------
# The plan
# --------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 6, 64), (7, 3, 5), (64, 8, 256), (1000, 4, 97), (1024, 4, 1),
                                   (1025, 4, 33), (3001, 6, 1000), (9000, 8, 1024), (5000, 1, 2)])
@pytest.mark.parametrize("holes", [False, True])
def test_plan(T, k, E, holes):
    g = np.random.default_rng(T + E)
    ids = torch.from_numpy(np.minimum(g.integers(0, E, (T, k)), g.integers(0, E, (T, k))).astype(np.int32))
    if holes and T:
        pick = torch.from_numpy(g.random((T, k)) < 0.3)
        ids[pick] = torch.from_numpy(g.choice([-1, E, E + 7, -(2 ** 31), 2 ** 31 - 1], int(pick.sum())).astype(np.int32))
    say("plan", T, k, E, holes)
    got = tg.route_plan(ids.cuda(), E)
    torch.cuda.synchronize()
    for x, y, name in zip(got, ref.plan(ids, E), ("offsets", "rows", "slots")):
        assert torch.equal(x.cpu(), y), name


def test_plan_of_one_expert_and_of_none():
    ids = torch.full((3000, 3), 5, dtype=torch.int32)
    for i in (ids, torch.full_like(ids, -1)):
        for x, y in zip(tg.route_plan(i.cuda(), 8), ref.plan(i, 8)):
            assert torch.equal(x.cpu(), y)


# --------------------------------------------------------------------------
# Rows to experts and back
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,D,R", [(1, 1, 8, 1), (5, 3, 72, 15), (33, 8, 520, 264), (200, 5, 2056, 1000)])
def test_gather_combine_and_gradients(dtype, T, k, D, R):
    g = torch.Generator().manual_seed(T)
    perm = torch.randperm(max(R, T * k), generator=g)[:T * k].view(T, k)
    slots = torch.where(perm < R, perm, torch.full_like(perm, -1)).to(torch.int32)
    if T > 2:
        slots[2, 0] = 2 ** 30
        slots[1] = -1                                 # a token without a row
    h, w, res = rand(1, R, D, dtype=dtype), rand(2, T, k), rand(3, T, D, dtype=dtype)
    dy = rand(4, T, D, dtype=dtype)
    ok = (slots >= 0) & (slots < R)
    at = slots.clamp(0, R - 1).long()
    wz = torch.where(ok, w.double(), torch.zeros(1, dtype=torch.float64))
    if T > 2:
        w[1, 0] = float("nan")                        # its weight has no row to weigh
    say("combine", dtype, T, k, D, R)
    picked = torch.where(ok[:, :, None], h.double()[at], torch.zeros(1, dtype=torch.float64))
    for weights, wt in ((w, wz), (None, ok.double())):
        for residual in (res, None):
            y = tg.expert_combine(h.cuda(), slots.cuda(), None if weights is None else weights.cuda(),
                                  residual=None if residual is None else residual.cuda())
            terms = picked * wt[:, :, None]
            want = terms.sum(1) + (0 if residual is None else residual.double())
            mag = terms.abs().sum(1) + (0 if residual is None else residual.double().abs())
            ref.assert_near(y, want, (k + 2) * 2.0 ** -24 * mag + ref.rounding(want, dtype) * 1.001, "combine")
    buf = res.cuda()
    tg.expert_combine(h.cuda(), slots.cuda(), residual=buf, out=buf)
    assert torch.equal(buf, tg.expert_combine(h.cuda(), slots.cuda(), residual=res.cuda()))

    dh0 = torch.full((R, D), 3.0, dtype=dtype, device="cuda")
    dh, dw = tg.expert_combine_backward(dy.cuda(), h.cuda(), slots.cuda(), w.cuda(), dh=dh0)
    torch.cuda.synchronize()
    want = torch.full((R, D), 3.0, dtype=torch.float64)
    want[at[ok]] = (dy.double()[:, None] * wz[:, :, None])[ok]
    ref.assert_near(dh, want, (2.0 ** -24 + ref.EPS[dtype]) * 1.001 * want.abs().clamp(min=ref.TINY[dtype]), "dh")
    terms = picked * dy.double()[:, None]
    ref.assert_near(dw, terms.sum(2), (D + 8) * 2.0 ** -24 * terms.abs().sum(2) + 1e-30, "dweights")

    x = rand(6, T, D, dtype=dtype)
    rows = torch.randint(-2, T + 2, (R,), generator=g).to(torch.int32)
    out = torch.full((R, D), 3.0, dtype=dtype, device="cuda")
    tg.expert_gather(x.cuda(), rows.cuda(), out=out)
    inside = (rows >= 0) & (rows < T)
    assert torch.equal(out.cpu(), torch.where(inside[:, None], x[rows.clamp(0, T - 1).long()], torch.tensor(3.0, dtype=dtype)))


def test_a_row_named_by_several_slots():
    """Elements of its gradient are each one of theirs, and their weights'
    gradients are right; other rows are as ever."""
    T, k, D, R = 40, 2, 1096, 50
    dy, h, w = rand(1, T, D, dtype=BF16), rand(2, R, D, dtype=BF16), rand(3, T, k)
    slots = torch.arange(T * k).view(T, k) % R
    slots[:, 1] = torch.where(torch.arange(T) < 30, torch.full((T,), 7), torch.full((T,), -1))
    slots = slots.to(torch.int32)
    dh, dw = tg.expert_combine_backward(dy.cuda(), h.cuda(), slots.cuda(), w.cuda(),
                                        dh=torch.zeros(R, D, dtype=BF16, device="cuda"))
    torch.cuda.synchronize()
    names = [[] for _ in range(R)]
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                names[int(slots[t, j])].append((w[t, j] * dy[t].float()).to(BF16))
    assert len(names[7]) == 30
    for r in range(R):
        if names[r]:
            assert bool((torch.stack(names[r]) == dh[r].cpu()).any(0).all()), r
        else:
            assert not dh[r].any()
    ok = slots >= 0
    terms = torch.where(ok[:, :, None], h.double()[slots.clamp(min=0).long()], torch.zeros(1, dtype=torch.float64)) * dy.double()[:, None]
    ref.assert_near(dw, terms.sum(2), (D + 8) * 2.0 ** -24 * terms.abs().sum(2) + 1e-30, "dweights")


def test_strided_rows_keep_what_is_around():
    T, k, D, R = 9, 2, 40, 18
    big = torch.full((R, D + 16), float("nan"), dtype=BF16, device="cuda")
    h = rand(1, R, D, dtype=BF16)
    big[:, 8:D + 8] = h.cuda()
    slots = torch.randperm(R, generator=torch.Generator().manual_seed(1)).view(T, k).to(torch.int32).cuda()
    w = rand(2, T, k).cuda()
    out = torch.full((T, D + 16), 5.0, dtype=BF16, device="cuda")
    tg.expert_combine(big[:, 8:D + 8], slots, w, out=out[:, 8:D + 8])
    assert torch.equal(out[:, 8:D + 8], tg.expert_combine(h.cuda(), slots, w))
    assert (out[:, :8] == 5).all() and (out[:, D + 8:] == 5).all()
    dy = rand(3, T, D, dtype=BF16).cuda()
    dbig = torch.full((R, D + 16), 5.0, dtype=BF16, device="cuda")
    dh, _ = tg.expert_combine_backward(dy, big[:, 8:D + 8], slots, w, dh=dbig[:, 8:D + 8])
    assert torch.equal(dh, tg.expert_combine_backward(dy, h.cuda(), slots, w)[0])
    assert (dbig[:, :8] == 5).all() and (dbig[:, D + 8:] == 5).all()


def test_sigmoid_far_out():
    """Logits whose sigmoids round to 0 or 1 in 32 bits are still chosen by
    their size."""
    x = torch.linspace(-120, 120, 50).view(1, 50)
    check_topk(x, 50, score="sigmoid", renormalize=False)
    assert math.isclose(float(tg.route_topk(x.cuda(), 1, score="sigmoid")[0]), 1.0)


def test_numbers_too_large_are_refused_before_memory_is_taken():
    x = rand(1, 4, 32).cuda()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for k in (33, 1 << 20, 1 << 40, (1 << 62) + 1):
        with pytest.raises(tg.TgemmError):
            tg.route_topk(x, k)
    for experts in (1025, 1 << 20, 1 << 40, (1 << 63) - 1):
        with pytest.raises(tg.TgemmError):
            tg.route_plan(ids, experts)
    assert torch.cuda.max_memory_allocated() == before
