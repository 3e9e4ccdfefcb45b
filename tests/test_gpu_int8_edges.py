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


# ------------------------------------------------------------- the product
def integer_rows(rng, M, N, K, cols, largest, kind):
    """Codes, weight codes and outliers whose products all are whole numbers, with the result: with
    scales of 127 and 127 a code's and a weight's unit are 1 (127 RN32(1/127) is 1)."""
    codes = rng.integers(-127, 128, (M, K)).astype(np.int8)
    CB = rng.integers(-127, 128, (N, K)).astype(np.int8)
    scale = np.full(M, 127, np.float32), np.full(N, 127, np.float32)
    if not cols:
        return codes, CB, scale, None, codes.astype(np.int64) @ CB.astype(np.int64).T
    codes[:, cols] = 0
    CB[:, cols] = rng.integers(-3, 4, (N, len(cols)))
    out = np.rint(rng.uniform(-largest, largest, (M, len(cols))))
    out[:, 0] = largest
    out = host(dev(out.astype(np.float32), DT[kind])).astype(np.int64)
    y = codes.astype(np.int64) @ CB.astype(np.int64).T + out @ CB[:, cols].astype(np.int64).T
    return codes, CB, scale, out, y


@pytest.mark.parametrize("M", [1, 16, 17, 40, 129, 300])
@pytest.mark.parametrize("K", [16, 208, 1040])
@pytest.mark.parametrize("largest,kind", [(0, "f16"), (300, "f16"), (40000, "f16"),
                                          (65504, "f16"), (3 << 16, "bf16"), (1 << 20, "bf16")])
def test_linear_whole_numbers(dq, M, K, largest, kind):
    """Sums of codes are exact up to K = 1040, and so they are beside outliers far above them: FP32
    results bit for bit.  (Everything is a whole number below 2^24.)"""
    rng = np.random.default_rng(M + K + largest)
    cols = [1, K - 3] if largest else []
    codes, CB, (scales, SCB), out, want = integer_rows(rng, M, 150, K, cols, largest, kind)
    assert np.abs(want).max() < 1 << 24
    rows = dq.Int8Rows(dev(codes), dev(scales))
    if cols:
        rows = rows._replace(cols=dev(np.array(cols)),
                             outliers=dev(out.astype(np.float32), DT[kind]))
    y = dq.int8_linear(rows, dev(CB), dev(SCB), out_dtype=torch.float32)
    assert np.array_equal(host(y), want), np.abs(host(y) - want).max()


@pytest.mark.parametrize("M", [8, 50])
@pytest.mark.parametrize("top", [300.0, 1000.0, 3000.0, 60000.0])
def test_linear_codes_beside_a_large_outlier(dq, M, top):
    """Results that take the codes alone (a weight of 0 at the outlier) keep 2^-21 of them; those
    that take both are FP32 sums of K / 16 steps beside it."""
    rng = np.random.default_rng(int(top))
    K, N = 1040, 130
    CB, SCB = weight(rng, N, K)
    x = rng.uniform(-1, 1, (M, K))
    x[:, 7], x[0, 7] = top * rng.uniform(0.5, 1, M), 0.0
    CB[::2, 7] = 0
    CB[1::4, 7] = 1
    rows = dq.int8_quantize(dev(x.astype(np.float32), torch.float16), 6.0, 8)
    y = dq.int8_linear(rows, dev(CB), dev(SCB), out_dtype=torch.float32)
    want, size = defs.linear(rows.codes.cpu().numpy(), host(rows.scales), CB, SCB,
                             rows.cols.cpu().numpy(), host(rows.outliers))
    tol = (2.0 ** -21 + np.where(CB[:, 7] != 0, K / 16 * 2.0 ** -23, 0)) * size
    assert (np.abs(host(y) - want) <= tol).all(), np.abs((host(y) - want) / size).max(0)


@pytest.mark.parametrize("M", [5, 60])
def test_linear_scales_far_from_one(dq, M):
    """Scales that only a caller's own rows have, beside outliers: of 0, negative, the smallest of
    the quantizer's and below; rows without a value above 0."""
    rng = np.random.default_rng(M)
    K, N = 96, 40
    CB, SCB = weight(rng, N, K)
    codes = rng.integers(-127, 128, (M, K)).astype(np.int8)
    scales = rng.uniform(0.5, 2, M).astype(np.float32)
    out = rng.normal(size=(M, 4)) * 20
    scales[0], scales[1], scales[2], scales[3] = 0.0, -1.5, 2.0 ** -100, 1e-35
    out[2:4] = out[2:4] * 1e-30
    scales[4], out[4] = 0.0, 0.0
    cols = np.array([0, 5, 64, 95])
    rows = dq.Int8Rows(dev(codes), dev(scales), dev(cols),
                       dev(out.astype(np.float32), torch.bfloat16))
    y = dq.int8_linear(rows, dev(CB), dev(SCB), out_dtype=torch.float32)
    want, size = defs.linear(codes, scales, CB, SCB, cols, host(rows.outliers))
    tol = (2.0 ** -21 + (K / 16 + 4) * 2.0 ** -23) * size
    assert (np.abs(host(y) - want) <= tol).all(), np.abs((host(y) - want) / (size + 1e-300)).max(1)


# ------------------------------------------------------------- equal runs of stages
def up256(n):
    return (n + 255) // 256 * 256


def steps_of(n):
    return -(-n // 64)


def width_of_runs(need, before, lanes, M, steps):
    """The tile width of a product whose CTAs take equal runs of stages, by the size of its
    workspace, which then has two parts of a tile for each CTA behind `before` bytes; else 0."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if need == before:
        return 0
    for width in (64, 128, 256):
        tiles = -(-M // width) * -(-lanes // 128)
        if need - before == min(tiles * (-(-steps // 2)), sms) * 2 * width * 128 * 4:
            return width
    raise AssertionError((need, before))


def linear_runs(dq, M, N, K, L):
    code_steps = steps_of(K) if L == 0 else (steps_of(K) + 1) // 2 * 2
    steps = code_steps + steps_of(L)
    before = 4096 + up256(N * steps_of(L) * 64) + up256(M * 4) + up256(M * steps * 128)
    need = dq.get_lib().dq4_int8_linear_workspace_bytes(M, N, K, L)
    return width_of_runs(need, before, N, M, steps)


def backward_runs(dq, M, N, K):
    need = dq.get_lib().dq4_int8_linear_backward_workspace_bytes(M, N, K)
    return width_of_runs(need, 4096, K, M, steps_of(N))


def gpu_weight(N, K, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    CB = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=gen)
    return CB, (0.5 + torch.rand(N, device="cuda", generator=gen)) * (4 / K ** 0.5)


def gpu_rows(dq, M, K, loud, seed, kind=torch.bfloat16, most=24):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=gen) * 0.8
    x[:, torch.randperm(K, device="cuda", generator=gen)[:loud]] *= 12
    return dq.int8_quantize(x.to(kind), 6.0 if loud else 0.0, most)


def test_counters_that_a_call_left_behind(dq):
    """A call whose wait ran out may leave counts of a tile's parts: the next one does without."""
    M, N, K = 60, 20000, 3008
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:  # (the shapes' plans)
        assert linear_runs(dq, M, N, K, 0) and backward_runs(dq, M, 22000, 3008)
    CB, SCB = gpu_weight(N, K, 1)
    rows = gpu_rows(dq, M, K, 0, 2)
    dy = torch.randn(M, 22000, device="cuda").half()
    W = gpu_weight(22000, 3008, 3)
    want = dq.int8_linear(rows, CB, SCB), dq.int8_linear_backward(dy, *W)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    for left in (1, 7):
        for call, is_ in ((lambda: dq.int8_linear(rows, CB, SCB, workspace=ws), want[0]),
                          (lambda: dq.int8_linear_backward(dy, *W, workspace=ws), want[1])):
            ws[:4096].view(torch.int32).fill_(left)
            for _ in range(2):
                assert torch.equal(call(), is_), left


# ------------------------------------------------------------- rows in 8 bits
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_quantize_thresholds_between_numbers(dq, kind):
    """A threshold means what it says: not the FP32 number next to it, which may be a value's own or
    0 (no threshold at all)."""
    rng = np.random.default_rng(7)
    x = rng.normal(size=(9, 200)) * 2
    x[3, 5], x[4, 6], x[5, 7] = 6.0, -6.0, 6.03125
    x[6] = 0
    x = dev(x.astype(np.float32), DT[kind])
    for threshold in (6.0 + 1e-9, 6.0 - 1e-9, 6.0, 1e-60, 5e-324, 1e-45, 6.03125 * (1 + 1e-15),
                      1e39, 1e300, 3.4028235677973366e38):
        rows = dq.int8_quantize(x, threshold, 128)
        codes, scales, cols, outliers, count = defs.quantize(host(x), threshold, 128)
        assert rows.count.item() == count, threshold
        assert np.array_equal(rows.cols.cpu().numpy(), cols), threshold
        assert np.array_equal(rows.codes.cpu().numpy(), codes), threshold
        assert np.array_equal(host(rows.scales), scales), threshold
        assert np.array_equal(host(rows.outliers), outliers), threshold
    for threshold in (-1e-60, -1.0, float("nan")):
        with pytest.raises(dq.Dq4Error):
            dq.int8_quantize(x, threshold)


@pytest.mark.parametrize("M", [1, 9, 24, 60])
def test_linear_codes_of_used_columns_leave_nothing(dq, M):
    """Codes of columns whose outliers are used do not count, however far above them they are: whole
    numbers, and outliers of 2^-20 of a code."""
    rng = np.random.default_rng(M)
    K, N, cols = 64, 33, [0, 9, 31, 32, 63]
    codes, CB = np.zeros((M, K), np.int8), rng.integers(-127, 128, (N, K)).astype(np.int8)
    codes[:, cols] = rng.integers(1, 128, (M, len(cols)))
    out = rng.integers(-100, 101, (M, len(cols))) * 2.0 ** -20
    rows = dq.Int8Rows(dev(codes), dev(np.full(M, 127, np.float32)), dev(np.array(cols)),
                       dev(out.astype(np.float32), torch.bfloat16))
    y = dq.int8_linear(rows, dev(CB), dev(np.full(N, 127, np.float32)), out_dtype=torch.float32)
    # (for many rows an outlier is two FP16 numbers, which end at 2^-24 of a unit)
    tol = 0 if M <= 16 else 2.0 ** -25 * np.abs(CB[:, cols].astype(int)).sum(1)
    assert (np.abs(host(y) - out @ CB[:, cols].T) <= tol).all()


@pytest.mark.parametrize("M", [3, 50])
@pytest.mark.parametrize("loud", [0, 3])
def test_linear_rows_near_the_largest_number(dq, M, loud):
    """Rows up to BF16's largest value through a weight that brings them back: no factor of the
    result is past FP32 on its way."""
    rng = np.random.default_rng(M + loud)
    K, N = 512, 70
    CB, SCB = weight(rng, N, K)
    SCB = (SCB * 1e-4).astype(np.float32)
    x = rng.uniform(-1, 1, (M, K)) * 2.0 ** 127 * (1 - 2.0 ** -9)
    if loud:
        x[:, loud:] *= 2.0 ** -20
    threshold = 2.0 ** 108 if loud else 0.0
    rows = dq.int8_quantize(dev(x.astype(np.float32), torch.bfloat16), threshold, 8)
    y = dq.int8_linear(rows, dev(CB), dev(SCB), out_dtype=torch.float32)
    want, size = defs.linear(rows.codes.cpu().numpy(), host(rows.scales), CB, SCB,
                             rows.cols.cpu().numpy() if loud else None,
                             host(rows.outliers) if loud else None)
    tol = (2.0 ** -21 + (K / 16 + 4) * 2.0 ** -23) * size
    assert np.isfinite(want.astype(np.float32)).all() and np.isfinite(host(y)).all()
    assert (np.abs(host(y) - want) <= tol).all()


def test_moe_rows_near_the_largest_number(dq):
    """Rows of 2^114 and inner values of 2^120 through weights that bring them back: sums of 512
    products with codes of 127, in the row's unit times that unit, would be past 2^128."""
    rng = np.random.default_rng(120)
    T, H, I, E = 5, 512, 32, 3
    x = dev((rng.uniform(0.5, 1, (T, H)) * 2.0 ** 114).astype(np.float32), torch.bfloat16)
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    w1[:], w2[:, ::2] = 127, 127
    s1[:, :I] *= np.float32(2.0 ** -114)
    s1[:, I:] *= np.float32(2.0 ** -6)
    s2 *= np.float32(2.0 ** -108)
    y = dq.int8_moe(x, logits, dev(w1), dev(s1), dev(w2), dev(s2), 2)
    want, _, _, size, unit = defs.moe(host(x), host(logits), w1, s1, w2, s2, 2, True)
    rounded_once(y, want, moe_off(unit, size, H, I), "bf16", "near the largest")


def close_on_gpu(y, rows, CB, SCB, bias, steps, u, what):
    """By the definition, in 64 bits on the GPU: for results too many for the host."""
    a = rows.codes.double() * (rows.scales.double()[:, None] / 127)
    if rows.cols is not None:
        for at, c in enumerate(rows.cols.tolist()):
            if c >= 0:
                a[:, c] = rows.outliers[:, at].double()
    w = CB.double() * (SCB.double()[:, None] / 127)
    want, size = a @ w.T, a.abs() @ w.abs().T
    if bias is not None:
        want, size = want + bias.double(), size + bias.double().abs()
    off = (y.double() - want).abs() - (2.0 ** -21 + steps * 2.0 ** -23) * size - u * want.abs()
    assert off.max() <= 2.0 ** -25, (what, off.max().item())


@pytest.mark.parametrize("N,K,L,few", [(4096, 4096, 0, 32), (4096, 4096, 5, 16), (4100, 512, 0, 16),
                                       (2048, 8192, 5, 32), (2064, 2048, 5, 16),
                                       (4096, 1024, 5, 32), (11008, 1024, 0, 16),
                                       (256, 16384, 0, 16), (256, 16368, 5, 32)])
def test_linear_on_both_sides_of_its_kernels(dq, N, K, L, few):
    """The change from the kernel for few rows, which needs no workspace, to that for many."""
    need = dq.get_lib().dq4_int8_linear_workspace_bytes
    CB, SCB = gpu_weight(N, K, N + K)
    for M in (16, 17, 32, 33):
        rows = gpu_rows(dq, M, K, L, M)
        most = 24 if L else 0
        assert (need(M, N, K, most) == 0) == (M <= few), M
        y = dq.int8_linear(rows, CB, SCB, out_dtype=torch.float32)
        close_on_gpu(y, rows, CB, SCB, None, K / 16 if L or K > 1040 else 0, 0, (M, N, K))


@pytest.mark.parametrize("M", [6, 14, 30, 60])
def test_linear_rows_that_are_no_number(dq, M):
    """A scale of NaN or an outlier that is not finite makes its row NaN, not infinite, and no
    other."""
    rng = np.random.default_rng(M)
    K, N = 144, 50
    CB, SCB = weight(rng, N, K)
    x = rng.normal(size=(M, K))
    x[:, 40] *= 30
    x[1, 3], x[2, 40], x[3, 40], x[4, 40] = np.nan, np.inf, -np.inf, np.nan
    for kind in ("f16", "bf16"):
        rows = dq.int8_quantize(dev(x.astype(np.float32), DT[kind]), 6.0, 16)
        y = host(dq.int8_linear(rows, dev(CB), dev(SCB), out_dtype=torch.float32))
        assert np.isnan(y[1:5]).all() and np.isfinite(y[[0, *range(5, M)]]).all()
        assert np.isnan(host(rows.scales)[1]) and np.isnan(host(rows.outliers)[4, 0])
        assert np.isinf(host(rows.outliers)[2:4, 0]).all()


def test_moe_weights_that_are_no_number(dq):
    """A NaN among a token's logits makes its weights and results NaN; a row without experts has
    weights of 0 and results of 0; no other token sees either."""
    rng = np.random.default_rng(5)
    T, H, I, E, k = 6, 32, 16, 5, 2
    logits = rng.normal(size=(T, E)).astype(np.float32)
    logits[1, 2], logits[3], logits[4, 1:] = np.nan, -np.inf, -np.inf
    for renormalize in (True, False):
        y, ids, weights = dq.int8_moe(
            dev(rng.normal(size=(T, H)).astype(np.float32), torch.bfloat16), dev(logits),
            *(dev(a) for a in weight(rng, E, 2 * I, H)), *(dev(a) for a in weight(rng, E, H, I)),
            k, renormalize, return_routing=True)
        assert y[1].isnan().all() and weights[1].isnan().all()
        assert (y[3] == 0).all() and (weights[3] == 0).all()
        assert y[[0, 2, 4, 5]].isfinite().all() and weights[[0, 2, 4, 5]].isfinite().all()
        assert weights[4].tolist() == [1.0, 0.0] and ids[4].tolist() == [0, 1]
        assert ids[3].tolist() == [0, 1]


def test_moe_most_experts_and_choices(dq):
    """The largest counts: 1024 experts, 256 tokens, 16 choices."""
    rng = np.random.default_rng(1024)
    T, H, I, E, k = 256, 16, 16, 1024, 16
    x = dev(rng.normal(size=(T, H)).astype(np.float32), torch.float16)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    logits[::3, 1000:] += 20  # (some experts with many tokens)
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    y, ids, weights = dq.int8_moe(x, dev(logits), dev(w1), dev(s1), dev(w2), dev(s2), k, False,
                                  return_routing=True)
    want, wids, wweights, size, unit = defs.moe(host(x), logits, w1, s1, w2, s2, k, False)
    assert np.array_equal(ids.cpu().numpy(), wids)
    # (the sum of 1024 terms: 32 a lane one after another, 5 steps over the lanes, 2^-24 each;
    # exponents to 32, rounded by 2^-24 of them; exp and the quotient)
    assert np.allclose(host(weights), wweights, rtol=2.0 ** -17, atol=0)
    off = moe_off(unit, size, H, I) + (2.0 ** -17 + k * 2.0 ** -24) * size
    rounded_once(y, want, off, "f16", "most")


# ------------------------------------------------------------- equal runs of stages
RUNS = [(60, 20100, 4112, 64), (61, 6177, 10000, 64), (250, 5000, 8000, 128),
        (100, 5000, 20000, 128), (500, 2500, 20000, 256), (509, 10995, 4080, 256)]


def by_runs(found, width):
    """Whether the plan is the one meant: a retuned one has to bring its own shapes here."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("shapes for 152 SMs")
    assert found == width


@pytest.mark.parametrize("M,N,K,width", RUNS)
@pytest.mark.parametrize("loud,kind", [(0, "f32"), (9, "f32"), (9, "bf16"), (5, "f16")])
def test_linear_in_runs(dq, M, N, K, width, loud, kind):
    """Tiles whose sums are cut where CTAs meet, at each width of a tile, ragged in every direction,
    with outlier columns; the same bits each time."""
    L = 24 if loud else 0
    by_runs(linear_runs(dq, M, N, K, L), width)
    CB, SCB = gpu_weight(N, K, M)
    rows = gpu_rows(dq, M, K, loud, N)
    bias = torch.randn(N, device="cuda").to(DT[kind]) if loud else None
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = dq.int8_linear(rows, CB, SCB, bias, DT[kind], bad=bad)
    close_on_gpu(y, rows, CB, SCB, bias, K / 16, {"f32": 2.0 ** -24, "bf16": 2.0 ** -8,
                                                  "f16": 2.0 ** -11}[kind], (M, N, K, kind))
    assert bad.item() == 0
    assert torch.equal(y, dq.int8_linear(rows, CB, SCB, bias, DT[kind]))


def backward_by_definition(dy, CB, SCB):
    w = ((CB.float() * SCB[:, None]) * torch.tensor(1 / 127, device="cuda")).to(dy.dtype).double()
    return dy.double() @ w, dy.double().abs() @ w.abs()


@pytest.mark.parametrize("M,N,K,width", [(60, 21992, 3008, 64), (60, 9112, 1168, 64),
                                         (500, 9936, 1072, 128), (300, 7744, 1376, 128),
                                         (500, 5416, 2640, 256), (2047, 5512, 4080, 256)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_backward_in_runs(dq, M, N, K, width, kind):
    by_runs(backward_runs(dq, M, N, K), width)
    CB, SCB = gpu_weight(N, K, M)
    dy = (torch.randn(M, N, device="cuda") * 0.05).to(DT[kind])
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx = dq.int8_linear_backward(dy, CB, SCB, bad=bad)
    want, size = backward_by_definition(dy, CB, SCB)
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    off = (dx.double() - want).abs() - (N / 16 + 4) * 2.0 ** -23 * size - u * want.abs()
    assert off.max() <= 2.0 ** -25 and bad.item() == 0
    assert torch.equal(dx, dq.int8_linear_backward(dy, CB, SCB))


# the product and a gradient, both in runs
BOTH = (60, 20100, 4112), (60, 21992, 3008)


@pytest.fixture(scope="module")
def in_runs(dq):
    (M, N, K), (m, n, k) = BOTH
    by_runs(linear_runs(dq, M, N, K, 24), 64)
    by_runs(backward_runs(dq, m, n, k), 64)
    W, V = gpu_weight(N, K, 1), gpu_weight(n, k, 2)
    rows = [gpu_rows(dq, M, K, 9, i) for i in range(4)]
    dys = [torch.randn(m, n, device="cuda").half() for _ in range(4)]

    def call(i, **more):
        return (dq.int8_linear(rows[i], *W, out_dtype=torch.bfloat16, **more),
                dq.int8_linear_backward(dys[i], *V, **more))
    want = [call(i) for i in range(4)]
    torch.cuda.synchronize()
    return call, want


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_runs_in_graphs_on_two_streams(dq, in_runs):
    call, want = in_runs
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(8):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            got = call(2)
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1]) and same(got, want[2])


def test_runs_from_threads(dq, in_runs):
    """Four host threads, two to a stream."""
    import threading
    call, want = in_runs
    streams = [torch.cuda.Stream() for _ in range(2)]
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i % 2]):
                for turn in range(8):
                    got = call((i + turn) % 4)
                    streams[i % 2].synchronize()
                    if not same(got, want[(i + turn) % 4]):
                        wrong.append((i, turn))
        except Exception as e:  # noqa: BLE001
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_runs_stay_in_their_workspace(dq, in_runs):
    """Workspaces of exactly the bytes that are asked for, full of anything, in the middle of larger
    buffers; a product and a gradient in turn through the same one."""
    call, want = in_runs
    lib, guard = dq.get_lib(), 1 << 16
    need = max(lib.dq4_int8_linear_workspace_bytes(*BOTH[0], 24),
               lib.dq4_int8_linear_backward_workspace_bytes(*BOTH[1]))
    buf = torch.full((need + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    for i in range(3):
        assert same(call(i, workspace=buf[guard:guard + need]), want[i])
    assert (buf[:guard] == 0xA5).all() and (buf[guard + need:] == 0xA5).all()


# ------------------------------------------------------------- as the README has it
@pytest.mark.parametrize("M", [7, 90])
def test_readme_function_trains_what_comes_before(dq, M):
    """The autograd function of the README: gradients of an adapter before a frozen weight, by the
    formula and by differences of the loss in 64 bits."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "class Frozen" in c]
    scope = {"torch": torch, "dq": dq}
    exec(code[0], scope)
    N, K, R = 96, 128, 8
    CB, SCB = gpu_weight(N, K, M)
    gen = torch.Generator("cuda").manual_seed(M)
    x = torch.randn(M, R, device="cuda", generator=gen)
    A = (torch.randn(R, K, device="cuda", generator=gen) * 0.5).requires_grad_()
    g = torch.randn(M, N, device="cuda", generator=gen).bfloat16()
    h = (x @ A).bfloat16()
    h.retain_grad()
    y = scope["Frozen"].apply(h, CB, SCB)
    assert torch.equal(y, dq.int8_linear(dq.int8_quantize(h.detach(), 6.0), CB, SCB,
                                         out_dtype=torch.bfloat16))
    (y.float() * g.float()).sum().backward()
    want, size = backward_by_definition(g, CB, SCB)
    off = (h.grad.double() - want).abs()
    assert (off <= 2.0 ** -8 * want.abs() + (N / 16 + 4) * 2.0 ** -23 * size).all()
    # A's own: x^T dh.  The loss is linear in A but for roundings, so a difference of it in 64 bits,
    # the weight as it is, is <dA, D>; the weight in BF16 and dh are off by 2^-8 of their terms each
    W = CB.double() * (SCB.double()[:, None] / 127)
    loss = lambda a: ((x.double() @ a) @ W.T * g.double()).sum()
    for _ in range(3):
        D = torch.randn(R, K, device="cuda", dtype=torch.float64, generator=gen)
        slope = (loss(A.detach().double() + D) - loss(A.detach().double() - D)) / 2
        reach = (x.double().abs().T @ (g.double().abs() @ W.abs()) * D.abs()).sum()
        assert ((A.grad.double() * D).sum() - slope).abs() <= (2.0 ** -7 + 2.0 ** -14) * reach


def test_single_rows_of_any_stride(dq):
    """A column turned into a row: its values follow one another, its stride to a next row is 1."""
    rng = np.random.default_rng(1)
    H, I, E = 1024, 32, 3
    x = dev(rng.normal(size=H).astype(np.float32), torch.bfloat16)
    row, view = x[None], x[:, None].t()
    assert view.stride() == (1, 1)
    args = (dev(rng.normal(size=(1, E)).astype(np.float32)),
            *(dev(a) for a in weight(rng, E, 2 * I, H)), *(dev(a) for a in weight(rng, E, H, I)), 2)
    assert torch.equal(dq.int8_moe(view, *args), dq.int8_moe(row, *args))
    for threshold in (0.0, 2.0):
        for a, b in zip(dq.int8_quantize(view, threshold), dq.int8_quantize(row, threshold)):
            assert a is b is None or torch.equal(a, b)
