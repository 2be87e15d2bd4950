"""Refusals of the log-probability and 4-bit entry points (no GPU needed)."""
import pytest
import torch

from linear_diffusion_cross_b200 import binding as B
from linear_diffusion_cross_b200 import build as _build
from linear_diffusion_cross_b200.logprob import FusedLinearLogProbs, fused_linear_logprobs
from linear_diffusion_cross_b200.w4 import W4Weight, linear_w4, quantize_w4

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return B.load()


def _x(n=4, d=32, dtype=BF):
    return torch.zeros(n, d, dtype=dtype)


def _tok(n=4):
    return torch.zeros(n, dtype=torch.int64)


def _w4(v=10, d=32, g=32):
    return W4Weight(torch.zeros(v, d // 2, dtype=torch.uint8),
                    torch.zeros(v, -(-d // g), dtype=BF), g)


def test_module_refusals():
    w = torch.zeros(10, 32, dtype=BF)
    for err, args, kw in [
        (ValueError, (_x(), _tok(), torch.zeros(10, 40, dtype=BF)), {}),
        (ValueError, (_x(), _tok(3), w), {}),
        (TypeError, (_x(), _tok().float(), w), {}),
        (TypeError, (_x(), _tok(), w.float()), {}),
        (TypeError, (_x(dtype=torch.float16), _tok(), w.half()), {}),
        (ValueError, (_x(), _tok(), w, torch.zeros(9, dtype=BF)), {}),
        (ValueError, (_x(), _tok(), w, torch.zeros(10)), {}),
        (ValueError, (_x(), _tok(), w), dict(top_k=21)),
        (ValueError, (_x(), _tok(), w), dict(top_k=11)),          # more than V
        (ValueError, (_x(), _tok(), w), dict(top_k=-1)),
        (RuntimeError, (_x(), _tok(), w), {}),                    # not on a GPU
        (ValueError, (_x(d=64), _tok(), _w4()), {}),
        (TypeError, (_x().float(), _tok(), _w4()), {}),
        (RuntimeError, (_x().requires_grad_(), _tok(), _w4()), {}),
    ]:
        with pytest.raises(err):
            fused_linear_logprobs(*args, **kw)
    with pytest.raises(ValueError):
        FusedLinearLogProbs(top_k=21)


def test_w4_refusals():
    with pytest.raises(ValueError):
        _w4(g=16)
    with pytest.raises(ValueError):
        _w4(d=48)
    with pytest.raises(TypeError):
        W4Weight(torch.zeros(10, 16, dtype=torch.int8), torch.zeros(10, 1, dtype=BF), 32)
    with pytest.raises(ValueError):
        W4Weight(torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(10, 2, dtype=BF), 32)
    with pytest.raises(ValueError):
        W4Weight(torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(10, 1), 32)
    with pytest.raises(ValueError):
        quantize_w4(torch.zeros(10, 40, dtype=BF))
    with pytest.raises(ValueError):
        quantize_w4(torch.zeros(10, 64, dtype=BF), group_size=48)
    with pytest.raises(TypeError):
        quantize_w4(torch.zeros(10, 64, dtype=torch.float16))
    with pytest.raises(RuntimeError):
        quantize_w4(torch.zeros(10, 64, dtype=BF))
    with pytest.raises(RuntimeError):
        linear_w4(_x(), _w4())
    with pytest.raises(TypeError):
        linear_w4(_x().float(), _w4())
    with pytest.raises(TypeError):
        linear_w4(_x(), _w4(), out_dtype=torch.float16)
    with pytest.raises(RuntimeError):
        linear_w4(_x().requires_grad_(), _w4())
    assert _w4(d=96, g=64).shape == (10, 96)


def _status(f, *a):
    with pytest.raises(B.FldceError) as e:
        f(*a)
    return e.value.status


def test_plan_refusals():
    for flags in (B.FLDCE_FLAG_SKIP_IGNORED, B.FLDCE_FLAG_FUSED_DH):
        h, _ = B.fldce_create(B.FLDCE_BF16, 64, 100, 10, flags=flags)
        assert _status(B.fldce_logprob_workspace_size, h, 1, 0) == B.FLDCE_ERR_UNSUPPORTED
        assert _status(B.fldce_logprob, h, B.make_logprob_call()) == B.FLDCE_ERR_UNSUPPORTED
        assert _status(B.fldce_logprob_bwd, h,
                       B.make_logprob_grad_call()) == B.FLDCE_ERR_UNSUPPORTED
        B.fldce_destroy(h)
    h, _ = B.fldce_create(B.FLDCE_BF16, 64, 100, 10, vocab_start=0, vocab_total=200)
    assert _status(B.fldce_logprob, h, B.make_logprob_call()) == B.FLDCE_ERR_UNSUPPORTED
    B.fldce_destroy(h)
    assert _status(B.fldce_logprob, None, B.make_logprob_call()) == B.FLDCE_ERR_INVALID_ARG
    assert _status(B.fldce_logprob_bwd, None,
                   B.make_logprob_grad_call()) == B.FLDCE_ERR_INVALID_ARG


# addresses that are never dereferenced: every call below is refused first
A = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), B.FLDCE_ERR_INVALID_ARG),
    (dict(N=11), B.FLDCE_ERR_INVALID_ARG),
    (dict(top_k=21), B.FLDCE_ERR_INVALID_ARG),
    (dict(top_k=-1), B.FLDCE_ERR_INVALID_ARG),
    (dict(top_k=2), B.FLDCE_ERR_INVALID_ARG),                 # no buffers for them
    (dict(H=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(W=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(w4=A, w4_scales=A, w4_group=32), B.FLDCE_ERR_INVALID_ARG),    # both weights
    (dict(token=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(W=None, w4=A, w4_scales=None, w4_group=32), B.FLDCE_ERR_INVALID_ARG),
    (dict(W=None, w4=A, w4_scales=A, w4_group=16), B.FLDCE_ERR_UNSUPPORTED),
    (dict(W=None, w4=A + 8, w4_scales=A, w4_group=32), B.FLDCE_ERR_ALIGN),
    (dict(H=A + 2), B.FLDCE_ERR_ALIGN),
    (dict(W=A + 8), B.FLDCE_ERR_ALIGN),
    (dict(bias=A + 2), B.FLDCE_ERR_ALIGN),
    (dict(token=A + 4), B.FLDCE_ERR_ALIGN),
    (dict(entropy=A + 2), B.FLDCE_ERR_ALIGN),
    (dict(workspace=None), B.FLDCE_ERR_WORKSPACE),
    (dict(workspace=A + 16), B.FLDCE_ERR_WORKSPACE),
    (dict(workspace_bytes=16), B.FLDCE_ERR_WORKSPACE),
])
def test_logprob_call_refusals(kw, code):
    h, _ = B.fldce_create(B.FLDCE_BF16, 64, 100, 10)
    args = dict(H=A, W=A, token=A, N=4, logprob=A, entropy=A, lse=A, workspace=A,
                workspace_bytes=1 << 40, stream=0)
    args.update(kw)
    assert _status(B.fldce_logprob, h, B.make_logprob_call(**args)) == code
    B.fldce_destroy(h)


def test_logprob_w4_needs_bf16_and_whole_groups():
    h, _ = B.fldce_create(B.FLDCE_FP32, 64, 100, 10)
    c = B.make_logprob_call(H=A, w4=A, w4_scales=A, w4_group=32, N=1, entropy=A, workspace=A,
                            workspace_bytes=1 << 40, stream=0)
    assert _status(B.fldce_logprob, h, c) == B.FLDCE_ERR_UNSUPPORTED
    B.fldce_destroy(h)
    h, _ = B.fldce_create(B.FLDCE_BF16, 72, 100, 10)
    assert _status(B.fldce_logprob, h, c) == B.FLDCE_ERR_UNSUPPORTED
    B.fldce_destroy(h)


@pytest.mark.parametrize("kw,code", [
    (dict(N=11), B.FLDCE_ERR_INVALID_ARG),
    (dict(dH=None, dW=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(H=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(lse=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(token=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(entropy=None), B.FLDCE_ERR_INVALID_ARG),
    (dict(db=A), B.FLDCE_ERR_INVALID_ARG),                    # without a bias
    (dict(dW=A + 8), B.FLDCE_ERR_ALIGN),
    (dict(dlogprob=A + 2), B.FLDCE_ERR_ALIGN),
    (dict(workspace=None), B.FLDCE_ERR_WORKSPACE),
    (dict(workspace_bytes=16), B.FLDCE_ERR_WORKSPACE),
])
def test_logprob_bwd_refusals(kw, code):
    h, _ = B.fldce_create(B.FLDCE_BF16, 64, 100, 10)
    args = dict(H=A, W=A, token=A, N=4, lse=A, entropy=A, dlogprob=A, dentropy=A, dH=A, dW=A,
                workspace=A, workspace_bytes=1 << 40, stream=0)
    args.update(kw)
    assert _status(B.fldce_logprob_bwd, h, B.make_logprob_grad_call(**args)) == code
    B.fldce_destroy(h)


def test_w4_call_refusals():
    q = B.fldce_w4_quantize
    assert _status(q, None, 0, 10, 64, 32, A, A, 0) == B.FLDCE_ERR_INVALID_ARG
    assert _status(q, A, 2, 10, 64, 32, A, A, 0) == B.FLDCE_ERR_UNSUPPORTED
    assert _status(q, A, 0, 10, 40, 32, A, A, 0) == B.FLDCE_ERR_UNSUPPORTED
    assert _status(q, A, 0, 0, 64, 32, A, A, 0) == B.FLDCE_ERR_INVALID_ARG
    assert _status(q, A, 0, 10, 64, 32, A + 4, A, 0) == B.FLDCE_ERR_ALIGN
    f = B.fldce_w4_linear
    assert _status(f, A, -1, A, A, 32, None, 10, 64, A, 0, None, 0) == B.FLDCE_ERR_INVALID_ARG
    assert _status(f, A, 1, A, A, 48, None, 10, 64, A, 0, None, 0) == B.FLDCE_ERR_UNSUPPORTED
    assert _status(f, A, 1, A, A, 32, None, 10, 64, A, 5, None, 0) == B.FLDCE_ERR_UNSUPPORTED
    assert _status(f, None, 1, A, A, 32, None, 10, 64, A, 0, None, 0) == B.FLDCE_ERR_INVALID_ARG
    assert _status(f, A + 2, 1, A, A, 32, None, 10, 64, A, 0, None, 0) == B.FLDCE_ERR_ALIGN
    assert _status(f, A, 1, A, A, 32, None, 10, 64, A + 2, 1, None, 0) == B.FLDCE_ERR_ALIGN


def test_workspace_grows_with_tokens_and_alternatives():
    h, _ = B.fldce_create(B.FLDCE_BF16, 2560, 151936, 1 << 30)
    size = B.fldce_logprob_workspace_size
    assert size(h, 0, 0) > 0
    assert size(h, 1, 0) < size(h, 1024, 0) < size(h, 1024, 1) < size(h, 1024, 20)
    # chunked: the size stays bounded however many tokens come
    assert size(h, 1 << 30, 20) < 1 << 30
    B.fldce_destroy(h)
