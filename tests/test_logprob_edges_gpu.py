"""Log-probabilities, alternatives and gradients where they are easily wrong:
frequent targets, cancelling products, masked weights, rows with nothing left
and long batches, against the 64-bit definitions of tests/_logprob_ref.py."""
import math

import pytest
import torch
import torch.utils.checkpoint

from linear_diffusion_cross_b200 import binding as B
from linear_diffusion_cross_b200.logprob import fused_linear_logprobs
from linear_diffusion_cross_b200.w4 import linear_w4, quantize_w4
from tests import _logprob_ref as R
from tests.test_logprob_gpu import close, grads_of, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("per,targets,D,chunk", [
    (5, 6, 72, 0), (8, 3, 72, 0), (5, 40, 264, 0), (8, 30, 72, 0), (64, 5, 1032, 0),
    (256, 3, 72, 0), (300, 1, 520, 0), (64, 12, 72, 256), (700, 2, 2056, 0)])
def test_rounding_is_given_back_to_frequent_targets(per, targets, D, chunk):
    """dW of targets that many tokens share: the target's element of a 16-bit G,
    nine tenths of the way to the middle between two 16-bit numbers, must not
    cost dW its rounding, whose sum over n tokens of either sign grows as fast
    as dW itself.  W is zero but for the targets (nearly flat: p = 1 / V)."""
    N, V = per * targets, 1500
    x, _, w, _ = make(N, D, V, BF, seed=N)
    g = torch.Generator(device=DEV).manual_seed(per)
    ids = torch.randperm(V, device=DEV, generator=g)[:targets]
    y = ids[torch.randperm(N, device=DEV, generator=g) % targets]
    keep = torch.zeros(V, 1, device=DEV, dtype=BF)
    keep[ids] = 1
    w = w * keep * 2.0 ** -6
    a = torch.full((N,), (1 + 0.9 * 2.0 ** -8) / (1 - 1 / V), device=DEV)
    a[torch.rand(N, device=DEV, generator=g) < 0.5] *= -1
    (_, got), _ = grads_of(x, y, w, None, 1.0, a, None, chunk_n=chunk)
    _, want, _, A = R.grads(x, y, w, None, 1.0, a, None)
    rest = A.clone()
    rest[torch.arange(N, device=DEV), y] = 0                     # what stays rounded
    u, dz, xa = 2.0 ** -8, R.bound_z(x, w, None, 1.0), x.double().abs()
    # fp32: p's relative error, every accumulation, the rest's own rounding
    fp = 4 * dz + 2.0 ** -18 + N * 2.0 ** -23
    lim = u * want.abs() + u * (1 + u) * (rest.T @ xa) + fp * (A.T @ xa) * (1 + u)
    err = (got.double() - want).abs()
    assert bool((err <= lim + 1e-30).all()), float((err / (lim + 1e-30)).max())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [2, 20, 40])
def test_a_cancelling_product_can_be_the_best(N, dtype):
    """Column 301's products 2^24 and -2^24 swallow its others in 32 bits (0
    instead of 1.40625); column 7's are small and sum to 0.5."""
    V, D = 600, 512
    x = torch.ones(N, D, device=DEV, dtype=dtype)
    w = torch.zeros(V, D, device=DEV)
    w[:, 1] = -10.0
    w[7, 1] = 0.5
    w[301] = 0.0
    small = [i for i in range(64, 256) if i % 64 < 32]
    w[301, small] = 1.875 * 2.0 ** -7
    w[301, 0], w[301, 256] = 2.0 ** 24, -(2.0 ** 24)
    w = w.to(dtype)
    r = fused_linear_logprobs(x, None, w, top_k=1)
    z = x.double() @ w.double().T
    assert torch.equal(r.top_ids[:, 0].long(), z.argmax(1)) and int(r.top_ids[0, 0]) == 301
    for k in (2, 3):
        r = fused_linear_logprobs(x, None, w, top_k=k)
        assert r.top_ids[:, :2].tolist() == [[301, 7]] * N


@pytest.mark.parametrize("k", [1, 5, 12, 20])
def test_near_ties_up_to_three_past_k_are_in_exact_order(k):
    """k + 3 logits that 32 bits cannot tell apart, above all others: exact ids
    from either side of the token count where the kernels change."""
    V, g = 900, torch.Generator(device=DEV).manual_seed(k)
    x = torch.ones(40, 16, device=DEV, dtype=BF)
    w = torch.zeros(V, 16, device=DEV)
    at = torch.randperm(V, device=DEV, generator=g)[:k + 3]
    w[at, 0] = 4096.0
    w[at, 1] = torch.arange(k + 3, device=DEV).float() * 2.0 ** -14
    w = w.to(BF)
    z = x.double() @ w.double().T
    ids = z.sort(dim=1, descending=True, stable=True).indices[:, :k].int()
    for n in (1, 9, 17, 32, 33, 40):
        r = fused_linear_logprobs(x[:n], None, w, top_k=k)
        assert torch.equal(r.top_ids, ids[:n]), n


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [4, 20, 40, 300])
def test_weights_of_minus_infinity(N, dtype):
    # logits of -inf without a bias: one in seven, and all of columns 256..511
    x, y, w, _ = make(N, 64, 1000, dtype, ignored=0.0)
    x = x.abs() + 0.125
    gone = torch.zeros(1000, dtype=torch.bool, device=DEV)
    gone[::7] = True
    gone[256:512] = True
    t = R.bounds(x, torch.where(gone[:, None], 0.0, w.float()), None, 1.0)
    w[gone, 3] = -math.inf
    r = fused_linear_logprobs(x, y, w, top_k=5)
    _, lp, ent, lse, ids, top = R.forward(x, y, w, None, 1.0, 5)
    close(r.lse, lse, t["lse"], "lse")
    close(r.logprob, lp, t["logprob"], "logprob")
    close(r.entropy, ent, t["entropy"], "entropy")
    assert torch.equal(r.top_ids, ids)
    close(r.top_logprobs, top, t["lse"], "top_logprobs")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("mask", ["lowest", -1e30, -1e9, -math.inf])
def test_rows_with_every_entry_masked_move_nothing(N, dtype, mask):
    # whatever value masks: the gradient is zero, not the NaN or the 2^100 that
    # exp(z - lse) gives where 32 bits cannot hold the difference
    x, y, w, b = make(N, 64, 600, dtype, bias=True, ignored=0.0)
    b[:] = torch.finfo(dtype).min if mask == "lowest" else mask
    a, e = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    got, r = grads_of(x, y, w, b, 1.0, a, e)
    for t in got:
        assert not t.any()
    assert not torch.isnan(r.entropy).any() and not torch.isnan(r.lse).any()


def test_fp32_tokens_beyond_a_grid_dimension():
    # 65535 tiles of 64 rows and some
    N, D, V = 65535 * 64 + 200, 8, 8
    x, y, w, b = make(N, D, V, F32, bias=True)
    r = fused_linear_logprobs(x, y, w, b, top_k=2)
    a = torch.randn(N, device=DEV)
    (gx, gw, gb), _ = grads_of(x, y, w, b, 1.0, a, None)
    for i in (slice(0, 300), slice(N - 300, N)):
        _, lp, ent, lse, ids, _ = R.forward(x[i], y[i], w, b, 1.0, 2)
        t = R.bounds(x[i], w, b, 1.0)
        close(r.lse[i], lse, t["lse"], "lse")
        close(r.logprob[i], lp, t["logprob"], "logprob")
        close(r.entropy[i], ent, t["entropy"], "entropy")
        assert torch.equal(r.top_ids[i], ids)
        dH, _, _, A = R.grads(x[i], y[i], w, b, 1.0, a[i], None)
        lim = R.grad_bounds(x[i], w, A, dH, dH.new_zeros(V, D), dH.new_zeros(V),
                            R.bound_z(x[i], w, b, 1.0), F32, 300)[0]
        assert bool(((gx[i].double() - dH).abs() <= lim).all())
    assert torch.isfinite(gw).all() and torch.isfinite(gb).all()


@pytest.fixture
def device_error():
    B.fldce_selftest_device_error(1)
    yield
    B.fldce_selftest_device_error(0)


@pytest.mark.parametrize("N", [3, 20, 40])
def test_a_wait_that_ran_out_gives_nan(N, device_error):
    # not sums of the stages that came, nor what the memory held before
    x, y, w, b = make(N, 64, 3001, BF, bias=True, ignored=0.0)
    w4 = quantize_w4(w, 32)
    e = torch.ones(N, device=DEV)
    for weight in (w, w4):
        for k in (0, 1, 8, 20):
            r = fused_linear_logprobs(x, y, weight, b, top_k=k)
            for t in (r.logprob, r.entropy, r.lse) + ((r.top_logprobs,) if k else ()):
                assert torch.isnan(t).all()
            assert k == 0 or ((r.top_ids >= -1) & (r.top_ids < 3001)).all()
    assert torch.isnan(linear_w4(x, w4)).all()
    got, _ = grads_of(x, y, w, b, 1.0, e, e)
    for t in got:
        assert torch.isnan(t).all()
    B.fldce_selftest_device_error(0)
    got, r = grads_of(x, y, w, b, 1.0, e, e, top_k=3)
    for t in (*got, *r):
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("flags", [0, B.FLDCE_FLAG_DW_FP32 | B.FLDCE_FLAG_DH_FP32])
def test_a_wait_that_ran_out_is_reported(N, flags, device_error):
    x, y, w, b = make(N, 64, 501, BF, bias=True, ignored=0.0)
    h, _ = B.fldce_create(B.FLDCE_BF16, 64, 501, N, flags=flags)
    nb = max(B.fldce_logprob_workspace_size(h, N, 2), B.fldce_logprob_bwd_workspace_size(h, N))
    ws = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    err = torch.zeros(2, dtype=torch.int32, device=DEV)
    lse, e = torch.zeros(N, device=DEV), torch.ones(N, device=DEV)
    t = F32 if flags else BF
    dH, dW, db = (torch.zeros(s, device=DEV, dtype=t) for s in ((N, 64), (501, 64), (501,)))
    B.fldce_logprob(h, B.make_logprob_call(H=x, W=w, bias=b, N=N, lse=lse, workspace=ws,
                                           workspace_bytes=nb, err_count=err))
    assert err.tolist() == [0, 1] and torch.isnan(lse).all()
    B.fldce_logprob_bwd(h, B.make_logprob_grad_call(
        H=x, W=w, bias=b, token=y, N=N, lse=e, entropy=e, dlogprob=e, dH=dH, dW=dW, db=db,
        workspace=ws, workspace_bytes=nb, err_count=err))
    assert err.tolist() == [0, 1]
    for g in (dH, dW, db):
        assert torch.isnan(g).all()
    B.fldce_destroy(h)


@pytest.mark.parametrize("N", [12, 40])
def test_rows_with_nan_are_nan_in_every_result(N):
    x, y, w, b = make(N, 64, 600, BF, bias=True, ignored=0.0)
    x[7, 3] = math.nan
    r = fused_linear_logprobs(x, y, w, b, top_k=3)
    for t in (r.logprob, r.entropy, r.lse, r.top_logprobs):
        assert torch.isnan(t[7]).all() and torch.isfinite(t[:7]).all()
    assert (r.top_ids[7] == -1).all()


@pytest.mark.parametrize("N", [6, 70])
def test_saved_tensor_hooks_and_checkpoints(N):
    x, y, w, b = make(N, 64, 700, BF, bias=True)
    e = torch.randn(N, device=DEV)
    want, _ = grads_of(x, y, w, b, 1.0, e, e)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    with torch.autograd.graph.save_on_cpu(pin_memory=True):
        r = fused_linear_logprobs(leaves[0], y, leaves[1], leaves[2])
    got = torch.autograd.grad([r.logprob, r.entropy], leaves, [e, e])
    for p, q in zip(got, want):
        assert torch.equal(p, q)

    def body(a, c, d):
        q = fused_linear_logprobs(a, y, c, d)
        return q.logprob, q.entropy

    out = torch.utils.checkpoint.checkpoint(body, *leaves, use_reentrant=False)
    got = torch.autograd.grad(out, leaves, [e, e])
    for p, q in zip(got, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("N", [6, 70])
def test_autograd_step_captured_in_a_graph(N):
    x, y, w, b = make(N, 64, 700, BF, bias=True)
    e = torch.randn(N, device=DEV)
    want, rw = grads_of(x, y, w, b, 1.0, e, e, top_k=2)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]

    def step():
        r = fused_linear_logprobs(leaves[0], y, leaves[1], leaves[2], top_k=2)
        return list(torch.autograd.grad([r.logprob, r.entropy], leaves, [e, e])) + [
            t.detach() for t in r]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, [*want, *(t.detach() for t in rw)]):
            assert torch.equal(p, q)
    # other inputs in the same buffers
    leaves[0].data.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    want, rw = grads_of(x.flip(0), y, w, b, 1.0, e, e, top_k=2)
    for p, q in zip(out, [*want, *(t.detach() for t in rw)]):
        assert torch.equal(p, q)


@pytest.mark.parametrize("N", [5, 90])
def test_an_ignore_index_inside_the_vocabulary(N):
    x, y, w, b = make(N, 64, 300, BF, bias=True, ignored=0.0)
    y[::2] = 0
    e = torch.randn(N, device=DEV)
    r = fused_linear_logprobs(x, y, w, b, ignore_index=0)
    z = torch.where(y == 0, -100, y)
    q = fused_linear_logprobs(x, z, w, b)
    for s, t in zip(r[:3], q[:3]):
        assert torch.equal(s, t)
    got, _ = grads_of(x, y, w, b, 1.0, e, e, ignore_index=0)
    want, _ = grads_of(x, z, w, b, 1.0, e, e)
    for s, t in zip(got, want):
        assert torch.equal(s, t)


@pytest.mark.parametrize("flags", [0, B.FLDCE_FLAG_DW_FP32 | B.FLDCE_FLAG_DH_FP32,
                                   B.FLDCE_FLAG_DW_ACCUMULATE])
@pytest.mark.parametrize("N,D,V,chunk", [(1, 72, 300, 0), (1, 1032, 40000, 0), (2, 264, 700, 0),
                                         (6, 2056, 5001, 0), (9, 136, 1501, 0), (16, 72, 4099, 0),
                                         (16, 4104, 700, 0), (47, 264, 700, 16)])
def test_few_tokens_gradients_are_rounded_once(N, D, V, chunk, flags):
    """One token's dW is a product of two numbers, and a peaked row's dH a few
    of W's rows: the rounding of a 16-bit G would be as large an error as the
    results' own.  G's two terms hold 2^-16."""
    x, y, w, b = make(N, D, V, BF, seed=V, sigma=4 / math.sqrt(D), bias=True, ignored=0.5)
    g = torch.Generator(device=DEV).manual_seed(N)
    a, e = torch.randn(N, device=DEV, generator=g), torch.randn(N, device=DEV, generator=g)
    r = fused_linear_logprobs(x, y, w, b)
    h, _ = B.fldce_create(B.FLDCE_BF16, D, V, N, chunk_N=chunk, flags=flags)
    nb = B.fldce_logprob_bwd_workspace_size(h, N)
    ws = torch.full((nb + 256,), 255, dtype=torch.uint8, device=DEV)
    fp32 = flags & B.FLDCE_FLAG_DW_FP32
    t = F32 if fp32 else BF
    dH = torch.zeros(N + 1, D, device=DEV, dtype=t)
    dW, db = torch.zeros(V, D, device=DEV, dtype=t), torch.zeros(V, device=DEV, dtype=t)
    B.fldce_logprob_bwd(h, B.make_logprob_grad_call(
        H=x, W=w, bias=b, token=y, N=N, lse=r.lse, entropy=r.entropy, dlogprob=a, dentropy=e,
        dH=dH, dW=dW, db=db, workspace=ws, workspace_bytes=nb))
    want = R.grads(x, y, w, b, 1.0, a, e)
    A = want[3]
    u = 2.0 ** -24 if fp32 else 2.0 ** -8
    eps = 2.0 ** -16 + 4 * R.bound_z(x, w, b, 1.0) + 2.0 ** -18
    xa, wa = x.double().abs(), w.double().abs()
    for got, ref, big, n in ((dH[:N], want[0], A @ wa, V), (dW, want[1], A.T @ xa, N),
                             (db, want[2], A.sum(0), N)):
        lim = u * ref.abs() + (eps + n * 2.0 ** -23) * big * (1 + u) + 1e-30
        err = (got.double() - ref).abs()
        assert bool((err <= lim).all()), float((err / lim).max())
    assert not dH[N].any() and (ws[nb:] == 255).all()
    B.fldce_destroy(h)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "w4"])
@pytest.mark.parametrize("N", [1, 20, 40])
def test_a_certain_tokens_logprob_is_as_good_as_its_rest(N, kind):
    """One logit far above the others: its log-probability is -(1 - p) for a 1 - p
    of about 1e-5, which a lse that is off like the fp32 logit (by 5e-6) would
    bury.  Only the rest's logits may be off like that."""
    D, V = 2048, 700
    x, _, w, _ = make(N, D, V, F32 if kind == "fp32" else BF, seed=N, sigma=0.01)
    w4 = None
    if kind == "w4":
        w4 = quantize_w4(w, 32)
        w = R.unpack(w4.packed, w4.scales, 32, F32)
    b = torch.zeros(V, device=DEV, dtype=x.dtype)
    b[333] = 18.0
    y = torch.full((N,), 333, device=DEV)
    r = fused_linear_logprobs(x, y, w4 if w4 is not None else w, b, top_k=1)
    _, lp, _, lse, ids, top = R.forward(x, y, w, b, 1.0, 1)
    assert torch.equal(r.top_ids, ids) and (ids == 333).all()
    rest = -torch.expm1(lp)                              # 1 - p
    tol = rest * (2 * R.bound_z(x, w, b, 1.0) + 2.0 ** -19) + 2.0 ** -23 * rest + 2.0 ** -45
    # The sum of exponentials is fp32 within a part of the vocabulary, and each
    # addition to one that holds the large term (1) is off by at most 2^-24: 16
    # in a 32-column chunk, 2 that join it, 4 chunks of a slice (the most; up to
    # 8 + 5 + 5 in the few-token kernel, one rounding in fp32).  Parts join in fp64.
    tol += 22 * 2.0 ** -24
    for got, want in ((r.logprob, lp), (r.top_logprobs[:, 0], top[:, 0])):
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("shift", [0.0, 1000.0])
@pytest.mark.parametrize("s", [1.0, -0.5])
def test_fp32_gradients_do_not_show_the_rounding_of_lse(shift, s):
    """Logits whose products and sums are exact in fp32 (multiples of 2^-6 below
    2^11), far from 0 and with one or two entries that make up most of a row:
    what is left is the rounding of probabilities, not that of lse (2^-15 at
    1000) or of lse log2(e)."""
    N, D, V = 24, 16, 40
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-2, 3, (N, D), device=DEV, generator=g).float()
    w = torch.randint(-64, 65, (V, D), device=DEV, generator=g).float() / 64
    b = torch.randint(-64, 65, (V,), device=DEV, generator=g).float() / 64 + shift / s
    y = torch.randint(0, V, (N,), device=DEV, generator=g)
    y[::3] = (s * (x @ w.T + b)).argmax(1)[::3]          # p near 1: a (1 - p) cancels
    a, e = torch.randn(N, device=DEV, generator=g), torch.randn(N, device=DEV, generator=g)
    got, _ = grads_of(x, y, w, b, s, a, e)
    want = R.grads(x, y, w, b, s, a, e)
    A = want[3]
    # p: exp 2^-22 and its argument, a difference (2^-24 of up to 2^6) scaled and
    # shifted (two roundings more, of as much); ln p the same; kap 2^-23, the
    # product and the sum with a 2^-23 more
    eps = 2.0 ** -22 + 3 * 64 * 2.0 ** -24 + 2.0 ** -22
    for t, ref, big, n in ((got[0], want[0], A @ w.double().abs(), V),
                           (got[1], want[1], A.T @ x.double().abs(), N), (got[2], want[2], A.sum(0), N)):
        # fp32 sums: at most 16 + n / 16 additions on a term's way
        lim = (eps + (17 + n / 16) * 2.0 ** -24) * big + 2.0 ** -24 * ref.abs() + 1e-30
        err = (t.double() - ref).abs()
        assert bool((err <= lim).all()), float((err / lim).max())


def test_lse_pair_writes_two_floats_a_row():
    x, y, w, b = make(37, 64, 900, F32, bias=True)
    lse = torch.full((37 * 2 + 3,), 7.0, device=DEV)
    h, _ = B.fldce_create(B.FLDCE_FP32, 64, 900, 37, flags=B.FLDCE_FLAG_LSE_PAIR)
    nb = B.fldce_logprob_workspace_size(h, 37, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    B.fldce_logprob(h, B.make_logprob_call(H=x, W=w, bias=b, N=37, lse=lse, workspace=ws,
                                           workspace_bytes=nb))
    assert (lse[74:] == 7.0).all()
    r = fused_linear_logprobs(x, y, w, b)
    assert torch.equal(lse[:37], r.lse) and r.lse.shape == (37,)
    assert bool((lse[37:74].abs() <= 2.0 ** -24 * lse[:37].abs()).all()) and lse[37:74].any()
    B.fldce_destroy(h)
