"""Attention over the 8-bit cache where values are no numbers; definitions and tolerances as in
test_gpu_attn."""

import numpy as np
import pytest
import torch

from tests.test_gpu_attn import Batch, check_attend, dq  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- values that are no numbers
@pytest.mark.parametrize("new", [1, 5, 60])
@pytest.mark.parametrize("dim,page,window", [(64, 16, 1000), (128, 16, 37), (128, 32, 999),
                                             (64, 32, 70), (64, 64, 129)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_codes_before_the_window_may_be_no_numbers(dq, new, dim, page, window, causal):
    """Pages that lie before every row's window hold another's codes, or none."""
    b = Batch(dq, [2000, 130, 75], 2, dim, page, seed=21)
    b.fill()
    for i, n in enumerate(b.lens):
        for j in range(max(0, n - new - window + 1) // page):
            for codes, scales in ((b.cache.k, b.cache.k_scale), (b.cache.v, b.cache.v_scale)):
                codes.view(torch.uint8)[int(b.table[i, j])] = 0x7F if j % 2 else 0xFF
                scales[int(b.table[i, j])] = 1.0 if j % 4 < 2 else float("nan")
    check_attend(dq, b, [new] * 3, 4, "bf16", causal, window)


@pytest.mark.parametrize("new", [1, 5, 60])
@pytest.mark.parametrize("dim,page,window", [(64, 16, 1000), (128, 16, 37), (128, 32, 999),
                                             (64, 32, 70), (64, 64, 129)])
def test_attend_pages_before_the_window_need_not_exist(dq, new, dim, page, window):
    """Their ids are not looked at: bad stays 0 (check_attend)."""
    b = Batch(dq, [2000, 130, 75], 2, dim, page, seed=22)
    b.fill()
    for i, n in enumerate(b.lens):
        before = max(0, n - new - window + 1) // page
        b.table[i, :before] = np.where(np.arange(before) % 2, -1, b.pages + 5)
        b.codes = [np.concatenate([c, np.full_like(c[:6], np.nan)]) if len(c) == b.pages else c
                   for c in b.codes]
        b.scales = [np.concatenate([s, np.full_like(s[:6], np.nan)]) if len(s) == b.pages else s
                    for s in b.scales]
    check_attend(dq, b, [new] * 3, 4, "bf16", True, window)
