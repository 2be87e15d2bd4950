"""The 4-bit head weight on the GPU: quantisation bit for bit, logits and
log-probabilities against 64 bits."""
import math

import pytest
import torch

from linear_diffusion_cross_b200.logprob import fused_linear_logprobs
from linear_diffusion_cross_b200.w4 import W4Weight, linear_w4, quantize_w4
from tests import _logprob_ref as R
from tests.test_logprob_gpu import check_forward, close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(N, D, V, group, seed=0, bias=False, sigma=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    sigma = 1.5 / math.sqrt(D) if sigma is None else sigma
    x = torch.randn(N, D, device=DEV, generator=g).to(BF)
    packed = torch.randint(0, 256, (V, D // 2), device=DEV, generator=g, dtype=torch.uint8)
    n = -(-D // group)
    scales = ((torch.rand(V, n, device=DEV, generator=g) + 0.5) * sigma / 4.6).to(BF)
    b = torch.randn(V, device=DEV, generator=g).to(BF) if bias else None
    y = torch.randint(0, V, (N,), device=DEV, generator=g)
    y[torch.rand(N, device=DEV, generator=g) < 0.2] = -100
    return x, y, W4Weight(packed, scales, group), b


def whole(w):
    return R.unpack(w.packed, w.scales, w.group_size)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,D,group", [(1, 32, 32), (7, 64, 128), (33, 96, 64), (100, 160, 128),
                                       (513, 1056, 32), (1000, 256, 64)])
def test_quantize(V, D, group, dtype):
    g = torch.Generator(device=DEV).manual_seed(V)
    w = (torch.randn(V, D, device=DEV, generator=g) * 0.02).to(dtype)
    if V > 6:
        w[3] = 0
        w[4, :5] = 1e-3
        w[4, 5:] = 0
        w[5] *= 1e-30
    q = quantize_w4(w, group)
    n = -(-D // group)
    f = torch.zeros(V, n * group, device=DEV)
    f[:, :D] = w.float()
    f = f.view(V, n, group)
    sc = (f.abs().amax(2) / 7).to(BF)
    assert torch.equal(q.scales, sc)
    s = sc.float()[:, :, None]
    qi = torch.where(s > 0, (f / s).round().clamp(-7, 7), torch.zeros_like(f)).view(V, -1)[:, :D]
    u = qi.to(torch.int32) & 15
    assert torch.equal(q.packed, (u[:, 0::2] | (u[:, 1::2] << 4)).to(torch.uint8))
    # and the weight it stands for is within half a step, or the clamp's share of 7 steps
    step = s.expand(V, n, group).reshape(V, -1)[:, :D].double()
    assert bool(((whole(q) - w.double()).abs() <= step * (0.5 + 7 * 2.0 ** -8) + 1e-37).all())


SHAPES = [(1, 32, 1, 32), (1, 64, 300, 128), (3, 96, 257, 64), (4, 256, 1000, 128),
          (5, 160, 513, 32), (8, 512, 4099, 64), (9, 1056, 333, 128), (16, 512, 5000, 32),
          (17, 2080, 700, 64), (31, 128, 2049, 128), (40, 416, 1111, 64), (130, 64, 600, 32),
          (2, 8224, 150, 128)]


@pytest.mark.parametrize("N,D,V,group", SHAPES)
@pytest.mark.parametrize("out", [F32, BF], ids=["fp32", "bf16"])
def test_linear(N, D, V, group, out):
    x, _, w, b = make(N, D, V, group, seed=V, bias=N % 2 == 1)
    got = linear_w4(x, w, b, out_dtype=out)
    assert got.shape == (N, V) and got.dtype == out
    wr = whole(w)
    ref = x.double() @ wr.T + (0 if b is None else b.double())
    tol = R.bound_z(x, wr, b, 1.0) + (2.0 ** -8 if out == BF else 2.0 ** -24) * ref.abs()
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("N,D,V,group", SHAPES)
def test_logprobs(N, D, V, group):
    x, y, w, b = make(N, D, V, group, seed=V + 1, bias=N % 2 == 0)
    for k, s in ((0, 1.0), (min(V, 1), -0.7), (min(V, 5), 0.5), (min(V, 20), 1.0)):
        check_forward(x, y, w, b, s, k, wref=whole(w))


def test_many_tokens():
    # several passes over the weight, several chunks of rows
    x, y, w, b = make(530, 96, 1111, 32, bias=True)
    check_forward(x, y, w, b, k=4, wref=whole(w))
    wr = whole(w)
    ref = x.double() @ wr.T + b.double()
    err = (linear_w4(x, w, b).double() - ref).abs()
    assert bool((err <= R.bound_z(x, wr, b, 1.0) + 2.0 ** -24 * ref.abs()).all())


def test_extreme_nibbles_and_scales():
    # every weight -8 (which quantize_w4 never writes), huge and tiny scales side by side
    V, D = 300, 128
    packed = torch.full((V, D // 2), 0x88, dtype=torch.uint8, device=DEV)
    scales = torch.full((V, 4), 2.0 ** -6, dtype=BF, device=DEV)
    scales[::2, 1] = 2.0 ** 10
    scales[1::3, 2] = 0
    w = W4Weight(packed, scales, 32)
    x = torch.ones(5, D, device=DEV, dtype=BF)
    ref = x.double() @ whole(w).T
    assert torch.equal(linear_w4(x, w).double(), ref)
    # one hot inputs read single weights: nibble order and group boundaries
    g = torch.Generator(device=DEV).manual_seed(0)
    w = W4Weight(torch.randint(0, 256, (V, D // 2), device=DEV, generator=g, dtype=torch.uint8),
                 (torch.rand(V, 4, device=DEV, generator=g) + 0.5).to(BF), 32)
    eye = torch.eye(D, device=DEV, dtype=BF)
    assert torch.equal(linear_w4(eye, w).double(), whole(w).T)


def test_ties_and_masks_in_4_bits():
    x, y, w, _ = make(6, 64, 900, 32)
    w = W4Weight(w.packed[:300].repeat(3, 1), w.scales[:300].repeat(3, 1), 32)
    check_forward(x, y, w, k=20, wref=whole(w))
    b = torch.zeros(900, device=DEV, dtype=BF)
    b[::2] = -math.inf
    check_forward(x, y, w, b, k=8, wref=whole(w))
    b[:] = -math.inf
    r = check_forward(x, y, w, b, k=2, wref=whole(w))
    assert (r.top_ids == -1).all()


def test_rows_past_the_call_stay():
    x, _, w, _ = make(12, 64, 301, 32)
    from linear_diffusion_cross_b200 import binding as B
    out = torch.full((12, 301), 7.0, device=DEV)
    err = torch.full((2,), 7, dtype=torch.int32, device=DEV)
    B.fldce_w4_linear(x, 5, w.packed, w.scales, 32, None, 301, 64, out, B.FLDCE_FP32, err)
    assert err.tolist() == [0, 0]
    assert (out[5:] == 7.0).all() and torch.equal(out[:5], linear_w4(x[:5], w))


def test_leading_dimensions_empty_and_views():
    x, y, w, b = make(12, 64, 301, 32, bias=True)
    ref = linear_w4(x, w, b)
    assert torch.equal(linear_w4(x.view(3, 4, 64), w, b), ref.view(3, 4, 301))
    assert torch.equal(linear_w4(x[0], w, b), linear_w4(x[:1], w, b)[0])
    assert linear_w4(x[:0], w, b).shape == (0, 301)
    half = W4Weight(w.packed[1:], w.scales[1:], 32)          # views off the 16-byte boundary
    assert torch.equal(linear_w4(x, half, b[1:]), ref[:, 1:])
    r = fused_linear_logprobs(x[:0], y[:0], w, b, top_k=1)
    assert r.top_ids.shape == (0, 1)


@pytest.mark.parametrize("N", [3, 20])
def test_captured_and_on_two_streams(N):
    x, y, w, b = make(N, 256, 3001, 64, bias=True)
    want = [linear_w4(x, w, b)] + list(fused_linear_logprobs(x, y, w, b, top_k=3))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [linear_w4(x, w, b)] + list(fused_linear_logprobs(x, y, w, b, top_k=3))
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)
    torch.cuda.synchronize()
    got = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(st):
            got += [[linear_w4(x, w, b)] + list(fused_linear_logprobs(x, y, w, b, top_k=3))
                    for _ in range(3)]
    torch.cuda.synchronize()
    for out in got:
        for p, q in zip(out, want):
            assert torch.equal(p, q)


def test_together():
    # a trained head is quantised once; its logits and its log-probabilities agree
    g = torch.Generator(device=DEV).manual_seed(2)
    head = (torch.randn(2000, 256, device=DEV, generator=g) * 0.1).to(BF)
    x = torch.randn(4, 256, device=DEV, generator=g).to(BF)
    y = torch.randint(0, 2000, (4,), device=DEV, generator=g)
    w = quantize_w4(head, 64)
    z = linear_w4(x, w)
    r = fused_linear_logprobs(x, y, w, top_k=1)
    tol = 2 * R.bounds(x, whole(w), None, 1.0)["lse"]
    close(r.lse, torch.logsumexp(z.double(), 1), tol, "lse")
    close(r.logprob, torch.log_softmax(z.double(), 1)[torch.arange(4), y], tol, "logprob")
    # the 16-bit head's results are near: half a 4-bit step per weight
    full = fused_linear_logprobs(x, y, head, top_k=1)
    err = (x.double().abs() @ (whole(w) - head.double()).abs().T).max()
    assert (r.lse - full.lse).abs().max() <= err + tol
    assert (r.logprob - full.logprob).abs().max() <= 2 * err + tol
