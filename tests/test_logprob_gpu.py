"""Token log-probabilities, entropy, alternatives and their gradients on the
GPU against the 64-bit definitions of tests/_logprob_ref.py, whose bounds are
the tolerances."""
import math
import threading

import pytest
import torch

from linear_diffusion_cross_b200 import binding as B
from linear_diffusion_cross_b200.logprob import FusedLinearLogProbs, fused_linear_logprobs
from linear_diffusion_cross_b200.module import fused_linear_cross_entropy_loss
from tests import _logprob_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(N, D, V, dtype, seed=0, sigma=None, bias=False, ignored=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    sigma = 1.5 / math.sqrt(D) if sigma is None else sigma
    x = torch.randn(N, D, device=DEV, generator=g).to(dtype)
    w = (torch.randn(V, D, device=DEV, generator=g) * sigma).to(dtype)
    b = torch.randn(V, device=DEV, generator=g).to(dtype) if bias else None
    y = torch.randint(0, V, (N,), device=DEV, generator=g)
    y[torch.rand(N, device=DEV, generator=g) < ignored] = -100
    return x, y, w, b


def close(got, want, tol, what):
    want = want.double()
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    lim = tol + 2.0 ** -24 * torch.where(same, 0.0, want.abs())      # the result's own rounding
    assert bool((err <= lim).all()), (what, float(err.max()), tol)


def check_forward(x, y, w, b=None, s=1.0, k=0, wref=None, **kw):
    wr = w if wref is None else wref
    r = fused_linear_logprobs(x, y, w, b, top_k=k, logit_scale=s, **kw)
    _, lp, ent, lse, ids, top = R.forward(x, y, wr, b, s, k)
    t = R.bounds(x, wr, b, s)
    if y is None:
        assert r.logprob is None
    else:
        close(r.logprob, lp, t["logprob"], "logprob")
    close(r.lse, lse, t["lse"], "lse")
    close(r.entropy, ent, t["entropy"], "entropy")
    if k:
        assert r.top_ids.dtype == torch.int32
        bad = (r.top_ids != ids).any(1).nonzero()
        assert bad.numel() == 0, (bad[:4], r.top_ids[bad[0]], ids[bad[0]])
        close(r.top_logprobs, top, t["lse"], "top_logprobs")
    else:
        assert r.top_ids is None and r.top_logprobs is None
    return r


@pytest.mark.parametrize("N,D,V,k,s,bias", [
    (1, 8, 1, 1, 1.0, False),
    (1, 64, 5, 5, 1.0, True),
    (2, 16, 255, 4, 0.5, False),
    (3, 72, 256, 1, 1.0, True),
    (7, 136, 257, 20, -0.7, False),
    (1, 512, 5000, 8, 1.0, False),
    (16, 128, 3001, 2, 2.0, True),
    (17, 264, 777, 0, 1.0, True),
    (32, 520, 4099, 20, 1.0, False),
    (33, 256, 1025, 3, -1.0, True),
    (64, 96, 33000, 8, 1.0, False),
    (257, 192, 2049, 20, 0.25, True),
    (300, 320, 40000, 5, 1.0, False),
    (515, 1032, 1000, 1, 1.0, False),
    (9, 4160, 600, 6, 1.0, False),
])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_forward(N, D, V, k, s, bias, dtype):
    x, y, w, b = make(N, D, V, dtype, seed=N + V, bias=bias)
    check_forward(x, y, w, b, s, k)


def test_forward_without_tokens_and_with_leading_dimensions():
    x, y, w, _ = make(24, 64, 500, BF)
    check_forward(x, None, w, k=3)
    r = FusedLinearLogProbs(top_k=3)(x.view(2, 3, 4, 64), y.view(2, 3, 4), w)
    q = fused_linear_logprobs(x, y, w, top_k=3)
    assert r.logprob.shape == r.entropy.shape == r.lse.shape == (2, 3, 4)
    assert r.top_ids.shape == r.top_logprobs.shape == (2, 3, 4, 3)
    for a, c in zip(r, q):
        assert torch.equal(a.reshape(-1), c.reshape(-1))
    one = fused_linear_logprobs(x[0], y[0], w, top_k=3)
    assert one.logprob.shape == () and one.top_ids.shape == (3,)
    assert torch.equal(one.top_ids, q.top_ids[0])


def test_no_tokens():
    x, y, w, b = make(0, 64, 500, BF, bias=True)
    r = fused_linear_logprobs(x, y, w, b, top_k=2)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 2)
    for t in (x, w, b):
        t.requires_grad_()
    r = fused_linear_logprobs(x, y, w, b)
    gx, gw, gb = torch.autograd.grad(r.logprob.sum() + r.entropy.sum(), (x, w, b))
    assert gx.shape == (0, 64) and not gw.any() and not gb.any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [2, 40])
def test_masked_entries(dtype, N):
    V = 700
    x, y, w, b = make(N, 64, V, dtype, bias=True, ignored=0.0)
    b[::3] = -math.inf                       # includes entries that are given tokens
    b[256:512] = -math.inf                   # a whole tile
    y[0] = 3
    check_forward(x, y, w, b, k=8)
    b[:] = -math.inf
    b[[5, 600]] = 1.0                        # two entries left, eight asked for
    r = check_forward(x, y, w, b, k=8)
    assert (r.top_ids[:, 2:] == -1).all()
    b[5] = -math.inf                         # one entry left: its p is 1
    r = check_forward(x, y, w, b, k=1)
    assert r.entropy.abs().max() <= 2.0 ** -20 and (r.top_ids == 600).all()
    b[:] = -math.inf                         # nothing left
    r = check_forward(x, y, w, b, k=2)
    assert (r.entropy == 0).all() and torch.isneginf(r.lse).all() and (r.top_ids == -1).all()


@pytest.mark.parametrize("N", [3, 50])
def test_lowest_value_bias(N):
    # fp32's lowest value instead of -inf: finite logits far below the others
    x, y, w, b = make(N, 64, 600, F32, bias=True, ignored=0.0)
    b[100:300] = torch.finfo(F32).min
    y[0] = 150
    r = fused_linear_logprobs(x, y, w, b, top_k=4)
    q = fused_linear_logprobs(x, y, w, torch.where(b < -1e30, -math.inf, b), top_k=4)
    assert torch.equal(r.lse, q.lse) and torch.equal(r.entropy, q.entropy)
    assert torch.equal(r.top_ids, q.top_ids)
    assert r.logprob[0] <= -3e38
    # every entry at it: the products' part is below its resolution, all equal
    b[:] = torch.finfo(F32).min
    r = fused_linear_logprobs(x, y, w, b)
    t = 2.0 ** -18 * math.log(600)
    assert (r.entropy - math.log(600)).abs().max() <= t


@pytest.mark.parametrize("N", [12, 20, 40])
def test_nan_rows_stay_their_own(N):
    x, y, w, b = make(N, 64, 600, BF, bias=True, ignored=0.0)
    ok = fused_linear_logprobs(x, y, w, b, top_k=3)
    x[7, 3] = math.nan
    x[9] = math.inf
    r = fused_linear_logprobs(x, y, w, b, top_k=3)
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[[7, 9]] = False
    for a, c in zip(r, ok):
        assert torch.equal(a[keep], c[keep])
    assert torch.isnan(r.lse[[7, 9]]).all() and torch.isnan(r.logprob[[7, 9]]).all()


@pytest.mark.parametrize("N", [4, 70])
def test_equal_logits_go_to_the_lowest_id(N):
    x, y, w, _ = make(N, 64, 1200, BF)
    check_forward(x, y, torch.zeros_like(w), k=20)           # ids 0..19
    w[300:] = w[:900].clone()                                        # every row of w again, 300 on
    check_forward(x, y, w, k=20)
    w[:] = w[:1]
    check_forward(x, y, w, k=7)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [2, 40])
def test_order_beyond_fp32(dtype, N):
    # logits 2^12 + j 2^-16 in a shuffled order: fp32 cannot tell them apart
    V = 600
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.ones(N, 16, device=DEV, dtype=dtype)
    w = torch.zeros(V, 16, device=DEV)
    w[:, 0] = 4096.0 if dtype == F32 else 4096.0
    # (j - 300) 2^-16 as two bf16 numbers
    j = (torch.randperm(V, device=DEV, generator=g) - 300).float()
    # columns 0..149 are the contenders; the others are clearly smaller
    w[150:, 0] = 0.0
    hi = (j / 16).floor() * 16
    w[:, 1] = hi * 2.0 ** -16
    w[:, 2] = (j - hi) * 2.0 ** -16
    w = w.to(dtype)
    y = torch.zeros(N, dtype=torch.int64, device=DEV)
    r = fused_linear_logprobs(x, y, w, top_k=1)
    z = x.double() @ w.double().T
    ids = z.sort(dim=1, descending=True, stable=True).indices
    # what the operator promises: candidates are found in fp32 (kept for the
    # best plus three), so the winner is exact among those it could tell apart
    top4 = z[:, :150].float().sort(dim=1, descending=True).values[:, 0]
    assert (z.gather(1, r.top_ids.long())[:, 0].float() == top4).all()
    # with at most as many contenders as candidates the order is exact
    w[4:150, 0] = 0
    z = x.double() @ w.double().T
    ids = z.sort(dim=1, descending=True, stable=True).indices.int()
    for k in (1, 3):
        r = fused_linear_logprobs(x, y, w, top_k=k)
        assert torch.equal(r.top_ids, ids[:, :k])


def grads_of(x, y, w, b, s, a, e, **kw):
    leaves = [t.detach().clone().requires_grad_() for t in (x, w)]
    bl = None if b is None else b.detach().clone().requires_grad_()
    r = fused_linear_logprobs(leaves[0], y, leaves[1], bl, logit_scale=s, **kw)
    outs, ups = [], []
    if a is not None:
        outs.append(r.logprob), ups.append(a)
    if e is not None:
        outs.append(r.entropy), ups.append(e)
    return torch.autograd.grad(outs, leaves + ([] if b is None else [bl]), ups), r


def check_grads(x, y, w, b, s, a, e, **kw):
    got, _ = grads_of(x, y, w, b, s, a, e, **kw)
    dH, dW, db, A = R.grads(x, y, w, b, s, a, e)
    dz = R.bound_z(x, w, b, s)
    lim = R.grad_bounds(x, w, A, dH, dW, db, dz, x.dtype, x.shape[0])
    for name, g, ref, t in zip(("dH", "dW", "db"), got, (dH, dW, db), lim):
        err = (g.double() - ref).abs()
        assert bool((err <= t).all()), (name, float((err / t).max()))
    return got


@pytest.mark.parametrize("N,D,V,s,bias,chunk", [
    (1, 8, 1, 1.0, False, 0),
    (1, 64, 300, 1.0, True, 0),
    (5, 72, 257, -0.8, True, 0),
    (16, 264, 777, 1.0, True, 0),
    (31, 96, 1501, -1.0, False, 0),
    (40, 96, 33001, 0.5, True, 32),
    (100, 136, 1003, 0.5, False, 0),
    (300, 256, 2000, 1.0, True, 128),
    (257, 520, 3001, 1.0, False, 100),
    (64, 1032, 5000, 1.0, True, 0),
])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_gradients(N, D, V, s, bias, chunk, dtype):
    x, y, w, b = make(N, D, V, dtype, seed=V, bias=bias)
    g = torch.Generator(device=DEV).manual_seed(3)
    a = torch.randn(N, device=DEV, generator=g)
    e = torch.randn(N, device=DEV, generator=g)
    check_grads(x, y, w, b, s, a, e, chunk_n=chunk)
    check_grads(x, y, w, b, s, a, None, chunk_n=chunk)
    check_grads(x, y, w, b, s, None, e, chunk_n=chunk)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_gradients_with_masked_entries(dtype):
    x, y, w, b = make(40, 64, 700, dtype, bias=True, ignored=0.2)
    b[::3] = -math.inf
    b[256:512] = -math.inf
    y[:20] = (y[:20].clamp_min(0) // 3) * 3 + 1          # not all on masked entries
    a, e = torch.randn(40, device=DEV), torch.randn(40, device=DEV)
    keep = torch.isfinite(b[y.clamp_min(0)]) | (y < 0)
    y = torch.where(keep, y, 1)
    got = check_grads(x, y, w, b, 1.0, a, e)
    masked = torch.isneginf(b)
    assert not got[1][masked].any() and not got[2][masked].any()
    b[:] = -math.inf                                     # rows that mean nothing move nothing
    got, _ = grads_of(x, y, w, b, 1.0, a, e)
    for t in got:
        assert not t.any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_ignored_tokens_move_nothing(dtype):
    x, y, w, _ = make(50, 64, 700, dtype, ignored=0.0)
    a = torch.randn(50, device=DEV)
    ref, _ = grads_of(x[:30], y[:30], w, None, 1.0, a[:30], None)
    y[30:] = -100
    y[40:] = 700                                         # out of range: like ignored
    y[45:] = -5
    a[30:] = math.nan                                    # never read
    got, r = grads_of(x, y, w, None, 1.0, a, None)
    assert not got[0][30:].any() and torch.equal(got[0][:30], ref[0])
    assert not r.logprob[30:].any()
    y[:] = -100
    got, _ = grads_of(x, y, w, None, 1.0, torch.ones_like(a), torch.zeros_like(a))
    assert not got[0].any() and not got[1].any()


def test_gradients_against_differences():
    x, y, w, b = make(6, 16, 40, F32, bias=True, sigma=0.4)
    a, e = torch.randn(6, device=DEV), torch.randn(6, device=DEV)
    got, _ = grads_of(x, y, w, b, 0.9, a, e)

    def f(xx, ww, bb):
        _, lp, ent, _, _, _ = R.forward(xx, y, ww, bb, 0.9)
        return float((a.double() * lp).sum() + (e.double() * ent).sum())

    base = [t.double() for t in (x, w, b)]
    h = 1e-5
    for i, g in enumerate(got):
        for j in (0, 7, g.numel() - 1):
            if j >= g.numel():
                continue
            hi, lo = [t.clone() for t in base], [t.clone() for t in base]
            hi[i].view(-1)[j] += h
            lo[i].view(-1)[j] -= h
            d = (f(*hi) - f(*lo)) / (2 * h)
            # central differences: error h^2 f''' / 6 + eps |f| / h, both below 1e-8 here
            assert abs(d - float(g.view(-1)[j])) <= 2e-5 * max(1.0, abs(d))


@pytest.mark.parametrize("N,V,chunk", [(9, 5000, 0), (150, 1500, 0), (150, 9000, 0),
                                       (700, 1999, 0), (300, 5000, 128)])
def test_targets_rounding_is_given_back(N, V, chunk):
    """The target's element of a 16-bit G, nine tenths of the way to the middle
    between two 16-bit numbers, must not cost dH and dW its rounding.  W is zero
    but for the targets, so that the rest of G hardly matters."""
    D = 72
    x, _, w, _ = make(N, D, V, BF, seed=N)
    ids = torch.randperm(V, device=DEV)
    y = ids[torch.arange(N, device=DEV) % (N // 2 + 1)]          # once or twice each
    y = y[torch.randperm(N, device=DEV)]
    keep = torch.zeros(V, 1, device=DEV, dtype=BF)
    keep[y] = 1
    w = w * keep * 2.0 ** -6                                     # nearly flat: p = 1 / V
    a = torch.full((N,), (1 + 0.9 * 2.0 ** -8) / (1 - 1 / V), device=DEV)
    got, _ = grads_of(x, y, w, None, 1.0, a, None, chunk_n=chunk)
    dH, dW, db, A = R.grads(x, y, w, None, 1.0, a, None)
    B_ = A.clone()
    B_[torch.arange(N, device=DEV), y] = 0                       # what stays rounded
    u, dz = 2.0 ** -8, R.bound_z(x, w, None, 1.0)
    xa, wa = x.double().abs(), w.double().abs()
    # fp32: p's relative error, every accumulation, the rest's own rounding
    fp = 4 * dz + 2.0 ** -18
    for t, want, big, small, n in ((got[0], dH, A @ wa, B_ @ wa, V), (got[1], dW, A.T @ xa, B_.T @ xa, N)):
        lim = u * want.abs() + u * (1 + u) * small + (fp + n * 2.0 ** -23) * big * (1 + u)
        err = (t.double() - want).abs()
        assert bool((err <= lim + 1e-30).all()), float((err / (lim + 1e-30)).max())


def test_only_the_gradients_asked_for():
    x, y, w, b = make(40, 64, 700, BF, bias=True)
    full, _ = grads_of(x, y, w, b, 1.0, torch.ones(40, device=DEV), None)
    for i in range(3):
        t = [x.clone(), w.clone(), b.clone()]
        t[i].requires_grad_()
        r = fused_linear_logprobs(t[0], y, t[1], t[2])
        assert not r.lse.requires_grad
        # an expanded upstream gradient (stride 0), as .sum() sends it
        (g,) = torch.autograd.grad(r.logprob.sum(), t[i])
        assert torch.equal(g, full[i])
    with pytest.raises(RuntimeError):
        x2 = x.clone().requires_grad_()
        r = fused_linear_logprobs(x2, y, w)
        (g,) = torch.autograd.grad(r.logprob.sum(), x2, create_graph=True)
        g.sum().backward()


def test_strided_and_unaligned_inputs():
    x, y, w, b = make(20, 64, 300, BF, bias=True)
    ref = fused_linear_logprobs(x, y, w, b, top_k=2)

    def odd(t):                                          # one element past a boundary
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    for xx, ww in ((odd(x), odd(w)), (x.T.contiguous().T, w.T.contiguous().T)):
        r = fused_linear_logprobs(xx, y.int() if ww is w else y, ww, odd(b), top_k=2)
        for p, q in zip(r, ref):
            assert torch.equal(p, q)
    r = fused_linear_logprobs(x, y.to(torch.int32), w, b, top_k=2)
    assert torch.equal(r.logprob, ref.logprob)
    xw = x.clone().requires_grad_()
    r = fused_linear_logprobs(xw.T.contiguous().T, y, w)
    (g1,) = torch.autograd.grad(r.logprob.sum(), xw)
    r = fused_linear_logprobs(xw, y, w)
    (g2,) = torch.autograd.grad(r.logprob.sum(), xw)
    assert torch.equal(g1, g2)


def test_results_do_not_depend_on_the_batch_for_ids():
    x, y, w, _ = make(300, 256, 5000, BF)
    whole = fused_linear_logprobs(x, y, w, top_k=8)
    t = 2 * R.bounds(x, w, None, 1.0)["lse"]
    for n in (1, 4, 31, 64):
        r = fused_linear_logprobs(x[:n], y[:n], w, top_k=8)
        assert torch.equal(r.top_ids, whole.top_ids[:n])
        close(r.lse, whole.lse[:n], t, "lse")


@pytest.mark.parametrize("N", [4, 300])
def test_same_results_every_time(N):
    x, y, w, b = make(N, 256, 9000, BF, bias=True)
    a, e = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    first = None
    for _ in range(3):
        got, r = grads_of(x, y, w, b, 1.0, a, e, top_k=8)
        now = list(got) + list(r)
        if first is not None:
            for p, q in zip(first, now):
                assert torch.equal(p, q)
        first = now


def _outs(N, k):
    return {"logprob": torch.full((N,), 77.0, device=DEV), "entropy": torch.full((N,), 77.0, device=DEV),
            "lse": torch.full((N,), 77.0, device=DEV),
            "ids": torch.full((N, k), 77, dtype=torch.int32, device=DEV),
            "top": torch.full((N, k), 77.0, device=DEV),
            "err": torch.full((2,), 77, dtype=torch.int32, device=DEV)}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [3, 45])
def test_c_call_writes_its_rows_only_and_counts_bad_tokens(dtype, n):
    x, y, w, _ = make(60, 64, 500, dtype, ignored=0.0)
    y[1] = 500
    y[2] = -1
    code = B.FLDCE_BF16 if dtype == BF else B.FLDCE_FP32
    h, _ = B.fldce_create(code, 64, 500, 60)
    nb = B.fldce_logprob_workspace_size(h, n, 4)
    ws = torch.full((nb + 256,), 171, dtype=torch.uint8, device=DEV)
    o = _outs(60, 4)
    B.fldce_logprob(h, B.make_logprob_call(
        H=x, W=w, token=y, N=n, top_k=4, logprob=o["logprob"], entropy=o["entropy"], lse=o["lse"],
        top_ids=o["ids"], top_logprobs=o["top"], workspace=ws, workspace_bytes=nb,
        err_count=o["err"]))
    assert o["err"].tolist() == [2, 0]
    for k in ("logprob", "entropy", "lse", "ids", "top"):
        assert (o[k][n:] == 77).all() and (o[k][:n] != 77).all()
    assert (ws[nb:] == 171).all()
    assert not o["logprob"][1:3].any()
    B.fldce_destroy(h)


@pytest.mark.parametrize("flags", [0, B.FLDCE_FLAG_DW_FP32, B.FLDCE_FLAG_DH_FP32,
                                   B.FLDCE_FLAG_DW_ACCUMULATE,
                                   B.FLDCE_FLAG_DW_ACCUMULATE | B.FLDCE_FLAG_DW_FP32])
@pytest.mark.parametrize("chunk", [0, 128])
def test_c_gradient_flags(flags, chunk):
    N, D, V = 300, 64, 500
    x, y, w, b = make(N, D, V, BF, bias=True)
    a, e = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    r = fused_linear_logprobs(x, y, w, b)
    h, _ = B.fldce_create(B.FLDCE_BF16, D, V, N, chunk_N=chunk, flags=flags)
    ws_bytes = B.fldce_logprob_bwd_workspace_size(h, N)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=DEV)
    dwt = F32 if flags & B.FLDCE_FLAG_DW_FP32 else BF
    dht = F32 if flags & B.FLDCE_FLAG_DH_FP32 else BF
    acc = 1.0 if flags & B.FLDCE_FLAG_DW_ACCUMULATE else 0.0
    dH = torch.full((N, D), 9.0, device=DEV, dtype=dht)
    dW = torch.full((V, D), 1.0, device=DEV, dtype=dwt)
    db = torch.full((V,), 1.0, device=DEV, dtype=dwt)
    err = torch.empty(2, dtype=torch.int32, device=DEV)
    B.fldce_logprob_bwd(h, B.make_logprob_grad_call(
        H=x, W=w, bias=b, token=y, N=N, lse=r.lse, entropy=r.entropy, dlogprob=a, dentropy=e,
        dH=dH, dW=dW, db=db, workspace=ws, workspace_bytes=ws_bytes, err_count=err))
    assert err.tolist() == [0, 0]
    rH, rW, rb, A = R.grads(x, y, w, b, 1.0, a, e)
    tH, tW, tb = R.grad_bounds(x, w, A, rH, rW + acc, rb + acc, R.bound_z(x, w, b, 1.0), BF, N)
    assert bool(((dH.double() - rH).abs() <= tH).all())
    assert bool(((dW.double() - acc - rW).abs() <= tW).all())
    assert bool(((db.double() - acc - rb).abs() <= tb).all())
    B.fldce_destroy(h)


@pytest.mark.parametrize("N", [4, 260])
def test_captured_graphs_and_streams(N):
    x, y, w, b = make(N, 128, 3000, BF, bias=True)
    a, e = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    ref, rref = grads_of(x, y, w, b, 1.0, a, e, top_k=3)
    h, _ = B.fldce_create(B.FLDCE_BF16, 128, 3000, N)

    def step(xx):
        r = fused_linear_logprobs(xx, y, w, b, top_k=3)
        dH, dW = torch.empty_like(xx), torch.empty_like(w)
        nb = B.fldce_logprob_bwd_workspace_size(h, N)
        ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
        B.fldce_logprob_bwd(h, B.make_logprob_grad_call(
            H=xx, W=w, bias=b, token=y, N=N, lse=r.lse, entropy=r.entropy, dlogprob=a, dentropy=e,
            dH=dH, dW=dW, workspace=ws, workspace_bytes=nb,
            stream=torch.cuda.current_stream()))
        return list(r) + [dH, dW]

    want = list(rref) + [ref[0], ref[1]]
    # two graphs, replayed in turn and at once on two streams
    xs = [x.clone(), x.clone()]
    graphs, outs = [], []
    for xx in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(xx))
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for out in outs:
            for p, q in zip(out, want):
                assert torch.equal(p, q)
    xs[1].zero_()
    graphs[1].replay()
    torch.cuda.synchronize()
    zero = step(torch.zeros_like(x))
    for p, q in zip(outs[1], zero):
        assert torch.equal(p, q)
    # eager calls on two streams at once
    got = []
    torch.cuda.synchronize()
    for st in streams:
        with torch.cuda.stream(st):
            got.append([step(x) for _ in range(3)])
    torch.cuda.synchronize()
    for runs in got:
        for out in runs:
            for p, q in zip(out, want):
                assert torch.equal(p, q)
    del graphs
    B.fldce_destroy(h)


@pytest.mark.parametrize("N", [4, 100])
def test_first_cuda_call_of_a_thread(N):
    # a new thread whose memory comes from the allocator's cache makes no CUDA
    # call before the library's: forward and backward work there all the same
    x, y, w, b = make(N, 128, 3000, BF, bias=True)
    a, e = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    ref, rref = grads_of(x, y, w, b, 1.0, a, e, top_k=3)
    h, _ = B.fldce_create(B.FLDCE_BF16, 128, 3000, N)
    nb = B.fldce_logprob_bwd_workspace_size(h, N)
    ws = torch.empty(max(nb, B.fldce_logprob_workspace_size(h, N, 0)), dtype=torch.uint8, device=DEV)
    dH, lse, ent = torch.zeros_like(x), torch.zeros(N, device=DEV), torch.zeros(N, device=DEV)
    torch.cuda.synchronize()
    calls = [
        lambda: B.fldce_logprob_bwd(h, B.make_logprob_grad_call(
            H=x, W=w, bias=b, token=y, N=N, lse=rref.lse, entropy=rref.entropy, dlogprob=a,
            dentropy=e, dH=dH, workspace=ws, workspace_bytes=nb)),
        lambda: B.fldce_logprob(h, B.make_logprob_call(
            H=x, W=w, bias=b, N=N, lse=lse, entropy=ent, workspace=ws, workspace_bytes=ws.numel()))]
    for call in calls:
        failed = []

        def body():
            try:
                call()
            except Exception as exc:
                failed.append(exc)

        th = threading.Thread(target=body)
        th.start()
        th.join()
        assert not failed, failed
        torch.cuda.synchronize()
    assert torch.equal(dH, ref[0]) and torch.equal(lse, rref.lse) and torch.equal(ent, rref.entropy)
    B.fldce_destroy(h)


def test_beside_the_loss():
    # the loss of the framework is minus the mean log-probability, with the same gradient
    x, y, w, b = make(200, 128, 3000, BF, bias=True)
    t = [v.clone().requires_grad_() for v in (x, w, b)]
    loss = fused_linear_cross_entropy_loss(t[0], y, t[1], t[2])
    g1 = torch.autograd.grad(loss, t)
    r = fused_linear_logprobs(t[0], y, t[1], t[2], top_k=4)
    n = int((y != -100).sum())
    own = -r.logprob.sum() / n
    g2 = torch.autograd.grad(own, t)
    assert abs(float(loss.detach()) - float(own.detach())) <= R.bounds(x, w, b, 1.0)["logprob"] + 2.0 ** -20
    a = torch.full((200,), -1.0 / n, device=DEV)
    dH, dW, db, A = R.grads(x, y, w, b, 1.0, a, None)
    lim = R.grad_bounds(x, w, A, dH, dW, db, R.bound_z(x, w, b, 1.0), BF, 200)
    for p, q, tol in zip(g1, g2, lim):
        assert bool(((p.double() - q.double()).abs() <= 2 * tol).all())


def test_calls_cut_into_chunks():
    # more tokens than the partial statistics of one chunk hold (1024 here)
    N, D, V = 1100, 8, 600000
    x, y, w, b = make(N, D, V, BF, bias=True)
    whole = fused_linear_logprobs(x, y, w, b, top_k=20)
    t = 2 * R.bounds(x, w, b, 1.0)["entropy"]
    for a, e in ((0, 5), (1000, 1100), (1030, 1031)):
        r = fused_linear_logprobs(x[a:e], y[a:e], w, b, top_k=20)
        assert torch.equal(r.top_ids, whole.top_ids[a:e])
        for p, q in zip(r, whole):
            if p.is_floating_point():
                close(p, q[a:e], t, "chunk")
    z, lp, ent, lse, ids, top = R.forward(x[1020:1040], y[1020:1040], w, b, k=20)
    assert torch.equal(whole.top_ids[1020:1040], ids)
    close(whole.lse[1020:1040], lse, t, "lse")


def test_every_token_count():
    # where kernels change with the number of tokens: 8, 16, 24, 32 and 256,
    # and below and above 128 KiB of hidden states
    x, y, w, b = make(300, 512, 1501, BF, bias=True)
    a, e = torch.randn(300, device=DEV), torch.randn(300, device=DEV)
    for n in (1, 7, 8, 9, 15, 16, 17, 23, 24, 25, 31, 32, 33, 63, 127, 128, 129, 255, 256, 257):
        check_forward(x[:n], y[:n], w, b, k=3)
        check_grads(x[:n], y[:n], w, b, 1.0, a[:n], e[:n])


def test_long_vocabulary_offsets():
    # a weight past 2^31 bytes and ids near its end
    D, V = 4096, 300000
    g = torch.Generator(device=DEV).manual_seed(5)
    w = torch.zeros(V, D, device=DEV, dtype=BF)
    w[-300:] = (torch.randn(300, D, device=DEV, generator=g) * 0.03).to(BF)
    x = torch.randn(40, D, device=DEV, generator=g).to(BF)
    y = torch.full((40,), V - 1, device=DEV)
    for n in (3, 40):
        r = fused_linear_logprobs(x[:n], y[:n], w, top_k=4)
        z = x[:n].double() @ w[-300:].double().T
        best = z.sort(dim=1, descending=True, stable=True)
        assert torch.equal(r.top_ids, best.indices[:, :4].int() + V - 300)
        lse = torch.log(z.exp().sum(1) + (V - 300))
        close(r.lse, lse, R.bounds(x, w[-300:], None, 1.0)["lse"], "lse")
        close(r.logprob, z[:, -1] - lse, R.bounds(x, w[-300:], None, 1.0)["logprob"], "logprob")
