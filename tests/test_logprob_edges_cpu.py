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
