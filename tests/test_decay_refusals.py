"""More refusals of the decayed attention, on the host before any CUDA call."""
import pytest

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from test_decay_host import FAKE, fwd


@pytest.fixture(scope="module")
def lib():
    la_build.build()
    return la.load()


@pytest.mark.parametrize("scale,want", [(1e-39, la.LA_ERR_ARG), (-1e-40, la.LA_ERR_ARG), (float("inf"), la.LA_ERR_ARG),
                                        (2e-38, la.LA_ERR_WORKSPACE), (-3e38, la.LA_ERR_WORKSPACE)])
def test_scales_are_normal_numbers(lib, scale, want):
    """The incoming state gradient is divided by `scale`, whose reciprocal has to be finite, and rows take its power of two."""
    a = [FAKE] * 8 + [None, None, None, 1, 4, 2, 4096, 64, 64, la.LA_BF16, scale, None, None, None, None, None, 0, None]
    assert lib.la_decay_bwd(*a) == want
    assert fwd(lib, scale=scale) == want
