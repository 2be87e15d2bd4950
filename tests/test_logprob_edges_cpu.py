"""Host-side edges of the log-probability and 4-bit entry points (no GPU needed)."""
import gc

import pytest
import torch
from torch.autograd import forward_ad

from linear_diffusion_cross_b200 import binding as B
from linear_diffusion_cross_b200 import build as _build
from linear_diffusion_cross_b200 import logprob
from linear_diffusion_cross_b200.logprob import fused_linear_logprobs
from linear_diffusion_cross_b200.module import (FusedLinearDiffusionCrossEntropyLoss,
                                                fused_linear_cross_entropy_loss)
from linear_diffusion_cross_b200.w4 import W4Weight, linear_w4

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return B.load()


def test_device_error_bits_are_checked():
    for bits in (-1, 256):
        with pytest.raises(B.FldceError):
            B.fldce_selftest_device_error(bits)
    B.fldce_selftest_device_error(0)


@pytest.mark.parametrize("dtype", [B.FLDCE_BF16, B.FLDCE_FP32])
@pytest.mark.parametrize("D,V,chunk", [(8, 3, 0), (80, 300, 0), (2560, 300, 0), (2560, 151936, 0),
                                       (4096, 32000, 1000), (512, 64, 0)])
def test_fewer_tokens_need_no_larger_workspace(D, V, chunk, dtype):
    # a workspace for the most tokens serves every call, as the loss's does
    h, _ = B.fldce_create(dtype, D, V, 1 << 20, chunk_N=chunk)
    ns = [0, 1, 8, 31, 32, 33, 100, 255, 256, 257, 512, 700, 768, 1024, 1280, 1281, 1536, 1700,
          2048, 2304, 3000, 4096, 10000, 65536, 1 << 20]
    for size in (lambda n: B.fldce_logprob_bwd_workspace_size(h, n),
                 lambda n: B.fldce_logprob_workspace_size(h, n, 0),
                 lambda n: B.fldce_logprob_workspace_size(h, n, min(V, 20))):
        got = [size(n) for n in ns]
        assert got == sorted(got), [(n, a, b) for n, a, b in zip(ns[1:], got, got[1:]) if b < a]
    B.fldce_destroy(h)


def _heads():
    w4 = W4Weight(torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(10, 1, dtype=BF), 32)
    y, p = torch.zeros(4, dtype=torch.int64), torch.ones(4)
    return {
        "logprobs": lambda x, w, b: fused_linear_logprobs(x, y, w, b).logprob,
        "logprobs-w4": lambda x, w, b: fused_linear_logprobs(x, y, w4, b).logprob,
        "linear-w4": lambda x, w, b: linear_w4(x, w4, b),
        "loss": lambda x, w, b: fused_linear_cross_entropy_loss(x, y, w, b),
        "loss-module": lambda x, w, b: FusedLinearDiffusionCrossEntropyLoss()(x, y, w, b, p_mask=p),
    }


@pytest.mark.parametrize("head", ["logprobs", "logprobs-w4", "linear-w4", "loss", "loss-module"])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_mode_is_refused(head, which):
    if which == 1 and "w4" in head:
        pytest.skip("no weight to differentiate")
    args = [torch.zeros(4, 32, dtype=BF), torch.zeros(10, 32, dtype=BF), torch.zeros(10, dtype=BF)]
    call = _heads()[head]
    with forward_ad.dual_level():
        dual = list(args)
        dual[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            call(*dual)
        with pytest.raises(RuntimeError, match="CUDA"):          # nothing dual: as ever
            call(*args)

    def f(t):
        return call(*(t if i == which else a for i, a in enumerate(args)))

    with pytest.raises(NotImplementedError):
        torch.func.jvp(f, (args[which],), (torch.ones_like(args[which]),))


def test_a_changing_scale_leaves_no_plans_behind(monkeypatch):
    alive = set()
    create, destroy = B.fldce_create, B.fldce_destroy

    def fldce_create(*a, **kw):
        h, n = create(*a, **kw)
        alive.add(h)
        return h, n

    def fldce_destroy(h):
        alive.remove(h)
        return destroy(h)

    monkeypatch.setattr(B, "fldce_create", fldce_create)
    monkeypatch.setattr(B, "fldce_destroy", fldce_destroy)
    logprob._plan.cache_clear()
    held = logprob._plan(BF, 64, 100, 1.0, -100, 0)
    assert logprob._plan(BF, 64, 100, 1.0, -100, 0) is held
    for i in range(300):
        p = logprob._plan(BF, 64, 100, 1.0 + i / 1000, -100, 0)
        assert p.workspace_size(5, 1) == B.fldce_logprob_workspace_size(p.handle, 5, 1)
        for n in range(20):
            assert p.bwd_workspace_size(n) == B.fldce_logprob_bwd_workspace_size(p.handle, n)
    gc.collect()
    assert len(alive) <= 66
    assert held.handle in alive                          # a graph may still need it
    with pytest.raises(B.FldceError):
        logprob._plan(BF, 64, 100, 0.0, -100, 0)
    logprob._plan.cache_clear()
    del p
    gc.collect()
    assert alive == {held.handle}
    for n in range(3000):
        held.workspace_size(n, 0)
    assert len(held._sizes) <= 1024
    del held
    gc.collect()
    assert not alive


def test_4_bit_weights_compare_by_identity():
    make = lambda: W4Weight(torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(10, 1, dtype=BF), 32)
    a, b = make(), make()
    assert a == a and a != b and a in [b, a] and len({a, b}) == 2


def test_scales_that_want_a_gradient_are_refused():
    x, y = torch.zeros(4, 32, dtype=BF), torch.zeros(4, dtype=torch.int64)
    w = W4Weight(torch.zeros(10, 16, dtype=torch.uint8),
                 torch.zeros(10, 1, dtype=BF).requires_grad_(), 32)
    for call in (lambda: linear_w4(x, w), lambda: fused_linear_logprobs(x, y, w)):
        with pytest.raises(RuntimeError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(RuntimeError, match="CUDA"):
            call()


def test_plans_with_a_pair_of_lse_are_for_log_probabilities():
    for kw in (dict(vocab_start=0, vocab_total=200), dict(flags=B.FLDCE_FLAG_SKIP_IGNORED),
               dict(flags=B.FLDCE_FLAG_FUSED_DH)):
        kw["flags"] = kw.get("flags", 0) | B.FLDCE_FLAG_LSE_PAIR
        with pytest.raises(B.FldceError):
            B.fldce_create(B.FLDCE_BF16, 64, 100, 10, **kw)
    h, _ = B.fldce_create(B.FLDCE_FP32, 64, 100, 10, flags=B.FLDCE_FLAG_LSE_PAIR)
    a = 1 << 20                                          # never dereferenced: refused first
    call = B.make_call(H=a, W=a, target=a, N=4, total=1.0, loss=a, workspace=a,
                       workspace_bytes=1 << 40, stream=0)
    with pytest.raises(B.FldceError) as e:
        B.fldce_forward_ex(h, call)
    assert e.value.status == B.FLDCE_ERR_UNSUPPORTED
    assert B.fldce_logprob_workspace_size(h, 4, 0) > 0
    B.fldce_destroy(h)
