"""Sizes at their ends, without a GPU: what the attention's kernels count in 32 bits is refused
past them, and a cache has heads."""

import pytest
import torch

from quantized_weight_dequantization_gb300 import KV8Cache
from tests.test_attn_abi import P, _cache, lib  # noqa: F401


@pytest.mark.parametrize("tokens,heads,kv", [
    (1 << 29, 8, 2), ((1 << 31) - 1, 2, 1), (1 << 25, 65408, 1), (1 << 32, 2, 2)])
def test_rows_of_a_kv_head(lib, tokens, heads, kv):  # noqa: F811
    status = lib.dq4_kv8_attention(_cache(kv_heads=kv), P, heads * 64, 64, 1, tokens, heads, P, 3,
                                   3, P, P, 2, 4, 0.1, 1, 0, P, None, P, 1 << 62, None, None)
    assert status == 2


def test_blocks_of_the_cache(lib):  # noqa: F811
    status = lib.dq4_kv8_attention(_cache(pages=1 << 30, kv_heads=2), P, 256, 64, 1, 5, 4, P, 3, 3,
                                   P, P, 2, 4, 0.1, 1, 0, P, None, P, 1 << 62, None, None)
    assert status == 2


def test_cache_without_heads():
    codes = torch.zeros((4, 0, 16, 64), dtype=torch.float8_e4m3fn)
    scales = torch.zeros((4, 0))
    with pytest.raises(ValueError, match="one kv head"):
        KV8Cache(codes, codes, scales, scales)
