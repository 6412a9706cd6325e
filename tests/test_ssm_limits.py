"""Sizes at the ends of the convolution's range: refused on the host where a kernel's 32-bit indexes would not hold them."""
import pytest

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

FAKE = 0x10000      # never dereferenced


@pytest.fixture(scope="module")
def lib():
    la_build.build()
    return la.load()


@pytest.mark.parametrize("E", [(1 << 31) - 8, (1 << 31) - 120])
def test_channels_past_the_last_whole_tile(lib, E):
    """The gradient's tiles of 128 channels: the last one's end has to be an int."""
    dt = la.LA_BF16
    assert lib.la_conv_workspace_size(1, 4, E, 4, dt) == 0
    assert lib.la_conv_bwd(FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None, None, None, None, 1, 4, E, 4, dt, dt, 1, None, None, FAKE,
                           1 << 62, None) == la.LA_ERR_ARG
    assert lib.la_conv_fwd(FAKE, FAKE, None, FAKE, None, None, None, 1, 4, E, 4, dt, dt, 1, None, None) == la.LA_ERR_ARG
    assert lib.la_conv_workspace_size(1, 4, (1 << 31) - 128, 4, dt) == 5 * ((1 << 31) - 128) * 4
