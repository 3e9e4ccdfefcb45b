"""The operators with 8-bit weights without a GPU: what test_int8_layers.py does not ask."""

import pytest

P = 1 << 12  # a fake aligned pointer, never followed on these paths
OK, N_, ALIGN, WORKSPACE = 0, 2, 6, 15


@pytest.fixture(scope="module")
def lib():
    from quantized_weight_dequantization_gb300 import build
    build.build()
    from quantized_weight_dequantization_gb300 import _int8
    return _int8._lib()


def test_moe_without_hidden_values(lib):
    """A token without values would still have choices and weights, which nothing would write."""
    def call(T, H, I):
        return lib.dq4_int8_moe(P, 64, 0, T, H, I, 8, P, 2, 1, P, P, P, P, P, P, P, P, 1 << 20, P,
                                None)
    assert call(4, 0, 32) == N_ and call(4, 64, 0) == N_ and call(4, 0, 0) == N_
    assert call(0, 0, 32) == OK and call(0, 64, 0) == OK


def test_thresholds_keep_their_side():
    """The library's FP32 threshold is the least that is not below the caller's, and never 0 for one
    that is not; negative ones and NaN stay what it refuses."""
    import math

    import numpy as np

    from quantized_weight_dequantization_gb300._int8 import _threshold
    for v in (6.0, 6.0 + 1e-9, 6.0 - 1e-9, 1e-60, 5e-324, 1e-45, 2.0 ** -149, 1e39, 1e300, math.inf,
              3.4028235677973366e38, 3.4028234663852886e38, 65504.1):
        f = _threshold(v)
        with np.errstate(over="ignore"):
            assert np.float32(f) == f and f >= v and f > 0, v
            assert float(np.nextafter(np.float32(f), np.float32(0))) < v, v
    assert all(_threshold(v) < 0 for v in (-1.0, -1e-60, -math.inf))
    assert math.isnan(_threshold(math.nan))


def test_moe_single_row_has_no_stride(lib):
    """The stride to a next row says nothing where there is none (the workspace is checked next)."""
    def call(T, stride, X=P):
        return lib.dq4_int8_moe(X, stride, 0, T, 64, 32, 8, P, 2, 1, P, P, P, P, P, P, P, None, 0,
                                P, None)
    assert call(1, 1) == call(1, 64) == call(2, 64) == WORKSPACE
    assert call(2, 1) == call(2, 68) == call(1, 1, P + 8) == ALIGN
