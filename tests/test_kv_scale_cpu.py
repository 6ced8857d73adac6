"""The attention's largest scale, without a GPU: the kernels multiply scores by scale * log2(e), which has to be
finite in FP32 (a row of scores 0 would be 0 x Inf)."""
import numpy as np
import pytest

from test_kv_cpu import _attention, lib  # noqa: F401  (the fixture)


@pytest.mark.parametrize("scale", [2.3587e38, 2.5e38, 3.0e38, 3.4028235e38])
def test_scales_whose_product_with_log2e_overflows_are_refused(lib, scale):  # noqa: F811
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(scale) * np.float32(1.4426950408889634))
    assert _attention(lib, scale=scale) == -3


def test_the_largest_scale_passes(lib):  # noqa: F811
    assert np.isfinite(np.float32(2.358e38) * np.float32(1.4426950408889634))
    assert _attention(lib, scale=2.358e38, out=None) == -1  # the next check
    assert _attention(lib, scale=1e-45, out=None) == -1
