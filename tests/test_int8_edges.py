"""The operators with 8-bit weights without a GPU: refusals that test_int8_layers.py does not have."""

import pytest

P = 1 << 12  # a fake aligned pointer, never followed on these paths
OK, N_ = 0, 2


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
