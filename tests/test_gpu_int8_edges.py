"""The operators with 8-bit weights on the GPU where their numbers are easiest lost, against the
64-bit definitions of oracle/int8_layers.py.  Tolerances as in test_gpu_int8_layers.py, but for
results that are held to the last bit: those say so.
"""

import numpy as np
import pytest
import torch

from oracle import int8_layers as defs
from tests.test_gpu_int8_layers import DT, dev, host, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_weight_dequantization_gb300 as m
    m.get_lib()
    return m


def rounded_once(got, want, off, kind, what):
    """got is what some value within `off` of want is rounded to: rounding keeps the order, so it
    lies between the ends' own.  (2^-30 of want: the ends go to 16 bits through FP32.)"""
    off = off + 2.0 ** -30 * np.abs(want)
    lo, hi = (host(torch.from_numpy(v).to(DT[kind])) for v in (want - off, want + off))
    got = host(got)
    out = (got < lo) | (got > hi) | ~np.isfinite(got)
    assert not out.any(), (what, int(out.sum()), out.size)


# ------------------------------------------------------------- mixture of experts
def moe_off(unit, size, H, I):
    """Before the results' own rounding: gate and up are FP32 sums of H / 16 steps, the inner
    values' two terms hold 2^-22 of them, sums of I / 16 steps, scales."""
    return unit * (H / 16 * 2.0 ** -23 + 2.0 ** -20) + size * (2.0 ** -22 + I / 16 * 2.0 ** -23
                                                               + 2.0 ** -19)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("I", [16, 48])
def test_moe_results_are_rounded_once(dq, kind, I):
    """Rows of one value, so that gate and up are one product each: what is lost of the inner
    values shows beside a result's rounding (11 bits of them alone: 1 to 2 % of the results)."""
    rng = np.random.default_rng(I)
    T, H, E = 256, 16, 2
    x = np.zeros((T, H))
    x[np.arange(T), rng.integers(0, H, T)] = rng.uniform(0.5, 2, T)
    x = dev(x.astype(np.float32), DT[kind])
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    y = dq.int8_moe(x, logits, dev(w1), dev(s1), dev(w2), dev(s2), 1)
    want, _, _, size, unit = defs.moe(host(x), host(logits), w1, s1, w2, s2, 1, True)
    rounded_once(y, want, moe_off(unit, size, H, I), kind, (kind, I))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("spread", [12, 18, 24, 27, 33])
def test_moe_small_inner_values_beside_large_ones(dq, kind, spread):
    """Inner values 2^spread below their row's largest, and results that take the small ones alone
    (codes of 0 at the others): held to 2^-22, or to 2^-39 of the row's largest."""
    rng = np.random.default_rng(spread)
    T, H, I, E = 19, 64, 96, 2
    x = dev(rng.normal(size=(T, H)).astype(np.float32), DT[kind])
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    s1[:, I:] *= 2.0 ** -spread  # of the rows of Wu,
    s1[:, I:I + 5] *= 2.0 ** spread  # all but a few places of one tile
    w2[:, 16:, :5] = 0
    s2[:, 16:] *= 2.0 ** spread
    y = dq.int8_moe(x, logits, dev(w1), dev(s1), dev(w2), dev(s2), 2)
    want, ids, weights, size, unit = defs.moe(host(x), host(logits), w1, s1, w2, s2, 2, True)
    floor = np.zeros_like(want)
    for t in range(T):
        for e, p in zip(ids[t], weights[t]):
            both = (w1[e] * (s1[e].astype(np.float64)[:, None] / 127)) @ host(x)[t]
            top = np.abs(both[:I] / (1 + np.exp(-both[:I])) * both[I:]).max()
            v = np.abs(w2[e].astype(np.float64)) * (s2[e].astype(np.float64)[:, None] / 127)
            floor[t] += p * 2.0 ** -39 * top * v.sum(1)
    rounded_once(y, want, moe_off(unit, size, H, I) + floor, kind, (kind, spread))


def test_moe_on_a_stream_of_its_own(dq):
    """What the call alone holds stays its own until the stream given is done with it, whatever the
    current stream allocates and writes meanwhile."""
    rng = np.random.default_rng(3)
    T, H, I, E, k = 8, 64, 32, 6, 2
    args = [dev(rng.normal(size=(T, H)).astype(np.float32), torch.float16),
            dev(rng.normal(size=(T, E)).astype(np.float32)),
            *(dev(a) for a in weight(rng, E, 2 * I, H)), *(dev(a) for a in weight(rng, E, H, I))]
    want = dq.int8_moe(*args, k)
    stream = torch.cuda.Stream()
    dq.int8_moe(*args, k, stream=stream)  # (the stream's workspace is there)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(stream):
            torch.cuda._sleep(20_000_000)  # (about 10 ms)
        y = dq.int8_moe(*args, k, stream=stream)
        others = [torch.full((T, k), 77, dtype=torch.int32, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert all((t == 77).all() for t in others)
        y, ids, weights = dq.int8_moe(*args, k, return_routing=True, stream=stream)
        stream.synchronize()
        assert torch.equal(y, want) and ids.shape == weights.shape == (T, k)
        assert torch.allclose(weights.sum(1), torch.ones(T, device="cuda"))
