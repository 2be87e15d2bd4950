"""Host-side edges of the log-probability and 4-bit entry points (no GPU needed)."""
import pytest

from linear_diffusion_cross_b200 import binding as B
from linear_diffusion_cross_b200 import build as _build


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
