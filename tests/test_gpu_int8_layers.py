"""The operators with 8-bit weights on the GPU against the 64-bit definitions of
oracle/int8_layers.py.

Tolerances, from the arithmetic.  u is half a step of the output type relative to its value.
 * quantize: bit for bit.
 * linear: sums of products of codes are exact below 2^24, above that FP32 sums of K / 16 steps
   (a step's rounding at most 2^-23 of the magnitudes); scales and the sum of the parts round five
   times: 2^-21 of the magnitudes; outlier values are exact to 2^-22.  Plus u |y|.
 * backward: products of 16-bit operands are exact, FP32 sums of N / 16 steps and four more.
 * moe: gate and up are FP32 sums of H / 16 steps, scales 2^-20; an error of theirs reaches y
   through `unit`; inner values are FP16 (2^-11) and FP32 sums of I / 16 steps; plus u |y|.
"""

import numpy as np
import pytest
import torch

from oracle import int8_layers as defs

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -149}


@pytest.fixture(scope="module")
def dq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_weight_dequantization_gb300 as m
    m.get_lib()
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    got, want = host(got), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
    fine = np.isfinite(want)
    over = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    assert not over.size or over.max() <= 0, (what, float(over.max()), int((over > 0).sum()))


def rows_of(rng, M, K, kind, loud=0):
    """Values of the type, as a device tensor, with a few loud columns."""
    x = rng.normal(size=(M, K)) * 0.8
    if loud:
        x[:, rng.permutation(K)[:loud]] *= 12
    return dev(x.astype(np.float32), DT[kind])


def weight(rng, *shape):
    codes = np.clip(np.rint(rng.normal(size=shape) * 32), -127, 127).astype(np.int8)
    scales = rng.uniform(0.5, 1.5, shape[:-1]) * (4 / np.sqrt(shape[-1]))
    return codes, scales.astype(np.float32)


# ------------------------------------------------------------- quantize
def check_quantize(dq, x, threshold, most, what):
    rows = dq.int8_quantize(x, threshold, most)
    codes, scales, cols, outliers, count = defs.quantize(host(x), threshold, most)
    assert np.array_equal(rows.codes.cpu().numpy(), codes), what
    assert np.array_equal(host(rows.scales), scales, equal_nan=True), what
    if threshold == 0:
        assert rows.cols is None and rows.outliers is None and rows.count is None
        return rows
    assert np.array_equal(rows.cols.cpu().numpy(), cols), what
    assert np.array_equal(host(rows.outliers), outliers, equal_nan=True), what
    assert rows.count.item() == count, what
    return rows


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 7), (9, 64), (8, 1000), (17, 1024), (5, 1032),
                                 (1, 4096), (4, 4104), (3, 14336), (2, 16384), (3, 16392),
                                 (2, 40000), (5, 5001), (700, 48)])
def test_quantize(dq, kind, M, K):
    rng = np.random.default_rng(M * 100003 + K)
    for loud in (0, min(3, K), min(K, 40)):
        x = rows_of(rng, M, K, kind, loud)
        for threshold, most in ((0.0, 64), (6.0, 2), (6.0, 128)):
            check_quantize(dq, x, threshold, most, (kind, M, K, loud, threshold, most))


def test_quantize_strides(dq):
    rng = np.random.default_rng(3)
    wide = rows_of(rng, 20, 3000, "bf16", 30)
    for view in (wide[:, :1024], wide[:, 8:2056], wide[:, 3:1003], wide[::3, :2048], wide[:, :0],
                 wide[:0], wide[2:3, 5:6], wide[5:6].expand(4, -1)):
        check_quantize(dq, view, 0.0, 64, tuple(view.shape))
        check_quantize(dq, view, 6.0, 16, tuple(view.shape))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_quantize_special_values(dq, kind):
    rng = np.random.default_rng(4)
    inf, nan = float("inf"), float("nan")
    x = host(rows_of(rng, 14, 264, kind))
    x[0] = 0
    x[1, 5] = nan
    x[2, 7] = inf
    x[3, 9] = -inf
    x[4] = 2.0 ** -24 if kind == "f16" else 2.0 ** -120
    x[5] = -0.0
    x[6, :] = 6.0  # all of them at the threshold
    x[7, 11], x[7, 12] = nan, inf
    x[8] = 65504 if kind == "f16" else 3e38
    x[9] = 0
    x[9, 3] = 2.0 ** -100 if kind == "bf16" else 2.0 ** -14
    x[10] = np.arange(264) / 2  # ties
    x[10, 0] = 127
    x = dev(x.astype(np.float32), DT[kind])
    for threshold in (0.0, 6.0, 1e-3, 70000.0, inf, 5.9990234375, 6.001):
        check_quantize(dq, x, threshold, 128, (kind, threshold))
        check_quantize(dq, x[:5], threshold, 1, (kind, threshold))


def test_quantize_leaves_its_workspace_ready(dq):
    rng = np.random.default_rng(5)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    for M, K, loud in ((40, 512, 9), (3, 96, 96), (900, 2048, 5), (2, 64, 0)):
        x = rows_of(rng, M, K, "f16", loud)
        rows = dq.int8_quantize(x, 6.0, 64, workspace=ws)
        want = defs.quantize(host(x), 6.0, 64)
        assert np.array_equal(rows.codes.cpu().numpy(), want[0])
        assert np.array_equal(rows.cols.cpu().numpy(), want[2])
        assert not ws.any()


# ------------------------------------------------------------- linear
def random_rows(dq, rng, M, K, loud, most=24, kind="f16"):
    x = rows_of(rng, M, K, kind, loud)
    return dq.int8_quantize(x, 6.0 if loud else 0.0, most)


def check_linear(dq, rows, CB, SCB, bias, kind, what, steps=0.0):
    b = None if bias is None else dev(bias.astype(np.float32), DT[kind])
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = dq.int8_linear(rows, dev(CB), dev(SCB), b, DT[kind], bad=bad)
    out = None if rows.outliers is None else host(rows.outliers)
    cols = None if rows.cols is None else rows.cols.cpu().numpy()
    want, size = defs.linear(rows.codes.cpu().numpy(), host(rows.scales), CB, SCB, cols, out,
                             None if b is None else host(b))
    tol = (2.0 ** -21 + steps) * size + U[kind] * np.abs(want) + TINY[kind]
    close(y, want, tol, what)
    assert bad.item() == 0, what
    return y


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 61, 64, 65, 127, 128, 129, 250, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (15, 64), (33, 80), (130, 320), (257, 1040),
                                 (129, 4096), (600, 528)])
def test_linear(dq, M, N, K):
    rng = np.random.default_rng(M * 1009 + N + K)
    CB, SCB = weight(rng, N, K)
    kinds = list(DT)
    for i, loud in enumerate((0, min(5, K))):
        kind = kinds[(M + N + i) % 3]
        rows = random_rows(dq, rng, M, K, loud, kind="bf16" if M % 2 else "f16")
        bias = rng.normal(size=N) if (M + i) % 2 else None
        check_linear(dq, rows, CB, SCB, bias, kind, (M, N, K, kind, loud))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (8, 1100, 11008), (40, 4096, 2048),
                                   (512, 1100, 4096), (1500, 2000, 1024), (700, 5000, 272)])
def test_linear_larger(dq, M, N, K):
    rng = np.random.default_rng(M + N + K)
    CB, SCB = weight(rng, N, K)
    for kind, loud in (("bf16", 0), ("f32", 17)):
        rows = random_rows(dq, rng, M, K, loud)
        check_linear(dq, rows, CB, SCB, rng.normal(size=N), kind, (M, N, K, kind))


@pytest.mark.parametrize("M", [3, 20, 70, 300])
def test_linear_extreme_codes(dq, M):
    """Sums up to 127^2 K: past 2^24 they are FP32 sums."""
    rng = np.random.default_rng(M)
    for K in (1024, 1040, 6000):
        CB = np.full((40, K), 127, np.int8)
        CB[1::2] = -127
        CB[2] = rng.choice([-127, 127], K)
        codes = np.full((M, K), -127, np.int8)
        codes[1] = rng.choice([-127, 127], K)
        rows = dq.Int8Rows(dev(codes), dev(np.full(M, 0.7, np.float32)))
        steps = 0.0 if K <= 1040 else K / 16 * 2.0 ** -23
        check_linear(dq, rows, CB, np.full(40, 1.3, np.float32), None, "f32", (M, K), steps)


@pytest.mark.parametrize("M", [2, 12, 40, 300])
def test_linear_columns(dq, M):
    """Columns that repeat, fall, or are out of range are not used and counted; codes of used
    columns are not; any number of columns up to 128."""
    rng = np.random.default_rng(M)
    K, N = 208, 45
    CB, SCB = weight(rng, N, K)
    codes = rng.integers(-127, 128, (M, K)).astype(np.int8)
    scales = rng.uniform(0.5, 2, M).astype(np.float32)
    out = rng.normal(size=(M, 128)) * 20
    for cols, wrong in (([3, 7, 7, 5, 200, 207, 208, -1, -2, -1], 4), ([-1] * 9, 0), ([0], 0),
                        (list(range(80, 208)), 0), ([1 << 40, 5], 1), ([-1, 9, -1, 63, 64], 0),
                        ([], 0)):
        o = dev(out[:, :len(cols)].astype(np.float32), torch.bfloat16)
        rows = dq.Int8Rows(dev(codes), dev(scales), dev(np.array(cols, np.int64)), o)
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = dq.int8_linear(rows, dev(CB), dev(SCB), out_dtype=torch.float32, bad=bad)
        want, size = defs.linear(codes, scales, CB, SCB, np.array(cols), host(o))
        close(y, want, 2.0 ** -21 * size + U["f32"] * np.abs(want), (M, cols))
        assert bad.item() == wrong, cols


@pytest.mark.parametrize("M", [4, 40])
def test_linear_outliers_far_from_the_codes(dq, M):
    """Rows of zeros but for their outliers, and outliers up to the type's largest value."""
    rng = np.random.default_rng(M)
    K, N = 320, 150
    CB, SCB = weight(rng, N, K)
    codes = rng.integers(-127, 128, (M, K)).astype(np.int8)
    scales = np.full(M, 0.4, np.float32)
    out = rng.normal(size=(M, 6)) * 10
    codes[0], scales[0] = 0, 0.0
    out[1] *= 5000.0
    out[2], scales[2] = out[2] * 1e30, 1e-20
    out[3] = 0
    rows = dq.Int8Rows(dev(codes), dev(scales), dev(np.array([0, 4, 63, 64, 200, 319])),
                       dev(out.astype(np.float32), torch.bfloat16))
    check_linear(dq, rows, CB, SCB, None, "f32", M, steps=2.0 ** -18)


@pytest.mark.parametrize("M", [5, 50])
def test_linear_not_finite(dq, M):
    rng = np.random.default_rng(M)
    K, N = 128, 70
    CB, SCB = weight(rng, N, K)
    x = host(rows_of(rng, M, K, "f16", 4))
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, 6] = -np.inf
    for threshold in (0.0, 6.0):
        rows = dq.int8_quantize(dev(x.astype(np.float32), torch.float16), threshold, 32)
        check_linear(dq, rows, CB, SCB, None, "bf16", threshold)


# ------------------------------------------------------------- backward
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (3, 24, 48), (16, 128, 64), (17, 136, 144),
                                   (65, 264, 320), (130, 64, 1040), (256, 1000, 272),
                                   (300, 2048, 512), (257, 72, 4096)])
def test_backward(dq, kind, M, N, K):
    rng = np.random.default_rng(M + N + K)
    CB, SCB = weight(rng, N, K)
    dy = dev((rng.normal(size=(M, N)) * 0.05).astype(np.float32), DT[kind])
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx = dq.int8_linear_backward(dy, dev(CB), dev(SCB), bad=bad)
    w = defs.weight16(CB, SCB, lambda f: torch.from_numpy(f).to(DT[kind]).float().numpy())
    want, size = defs.linear_backward(host(dy), w)
    tol = (N / 16 + 4) * 2.0 ** -23 * size + U[kind] * np.abs(want) + TINY[kind]
    close(dx, want, tol, (kind, M, N, K))
    assert bad.item() == 0


# ------------------------------------------------------------- mixture of experts
def check_moe(dq, x, logits, w1, s1, w2, s2, top_k, renormalize, kind, what):
    y, ids, weights = dq.int8_moe(x, logits, dev(w1), dev(s1), dev(w2), dev(s2), top_k,
                                  renormalize, return_routing=True)
    want, wids, wweights, size, unit = defs.moe(host(x), host(logits), w1, s1, w2, s2, top_k,
                                                renormalize)
    assert np.array_equal(ids.cpu().numpy(), wids), what
    # the exponent d = logit - largest is rounded to FP32, by up to 2^-24 |d|, which moves exp(d)
    # by that factor of itself; results below 2^-126 have steps of 2^-149, so exp(-200) is 0
    row = host(logits)
    with np.errstate(invalid="ignore"):
        d = np.abs(np.take_along_axis(row, wids.astype(np.int64), 1) - row.max(1, keepdims=True))
    d = np.where(np.isfinite(d), d, 0)
    close(weights, wweights, (2.0 ** -20 + 2.0 ** -24 * d) * np.abs(wweights) + 2.0 ** -148, what)
    H, I = x.shape[1], w2.shape[2]
    tol = (unit * (H / 16 * 2.0 ** -23 + 2.0 ** -20)
           + size * (2.0 ** -11 + I / 16 * 2.0 ** -23 + 2.0 ** -19) + U[kind] * np.abs(want)
           + TINY[kind])
    close(y, want, tol, what)
    return y


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 23, 33, 70, 256])
@pytest.mark.parametrize("H,I,E,k", [(16, 16, 1, 1), (64, 32, 4, 2), (272, 48, 8, 3),
                                     (128, 336, 60, 6), (1040, 64, 5, 5), (80, 16, 130, 16)])
def test_moe(dq, T, H, I, E, k):
    rng = np.random.default_rng(T + H + I + E)
    kind = "bf16" if (T + E) % 2 else "f16"
    x = rows_of(rng, T, H, kind, 1)
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    check_moe(dq, x, logits, w1, s1, w2, s2, k, T % 2 == 0, kind, (T, H, I, E, k))


def test_moe_routing(dq):
    """Ties, NaN, infinities, masked experts, rows whose mask leaves nothing."""
    rng = np.random.default_rng(8)
    T, H, I, E = 14, 64, 32, 40
    logits = rng.integers(-2, 3, (T, E)).astype(np.float32)
    inf, nan = np.inf, np.nan
    logits[1] = -inf
    logits[2, 5:] = -inf
    logits[3, 2:] = -inf
    logits[4] = 0
    logits[5] = -0.0
    logits[5, 1::2] = 0.0
    logits[6, 7] = nan
    logits[7] = -3.4028235e38
    logits[7, 39] = -inf
    logits[8] = 1e-45
    logits[9] = nan
    logits[10] = 3.4028235e38
    logits[10, 33] = 0
    logits[11] = 200 * logits[11]
    x = rows_of(rng, T, H, "bf16")
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    for k in (1, 4, 16):
        for renormalize in (True, False):
            check_moe(dq, x, dev(logits), w1, s1, w2, s2, k, renormalize, "bf16", (k, renormalize))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_moe_scales(dq, kind):
    """Rows far from 1 in both directions, rows of zeros, strided rows, and values that are no
    numbers, which stay in their token."""
    rng = np.random.default_rng(9)
    T, H, I, E = 7, 96, 48, 6
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    s2[3] *= 0
    wide = host(rows_of(rng, T, H + 40, kind))
    x = wide[:, 8:8 + H]
    x[0] *= 2.0 ** -10 if kind == "f16" else 2.0 ** -60
    x[1] *= 2.0 ** 10 if kind == "f16" else 2.0 ** 30
    x[2] = 0
    x[3, 1:] = 0
    logits = rng.normal(size=(T, E)).astype(np.float32)
    view = dev(wide.astype(np.float32), DT[kind])[:, 8:8 + H]
    s2 = s2 * (2.0 ** -20 if kind == "f16" else 1)
    check_moe(dq, view, dev(logits), w1, s1, w2, s2, 3, True, kind, kind)
    bad = view.clone()
    bad[4, 2], bad[5, 3] = float("nan"), float("inf")
    y = dq.int8_moe(bad, dev(logits), dev(w1), dev(s1), dev(w2), dev(s2), 3)
    was = dq.int8_moe(view, dev(logits), dev(w1), dev(s1), dev(w2), dev(s2), 3)
    assert y[4:6].isnan().all()
    keep = [0, 1, 2, 3, 6]
    assert torch.equal(y[keep], was[keep])


def test_moe_same_expert_for_all(dq):
    rng = np.random.default_rng(10)
    T, H, I, E = 61, 128, 64, 9
    x = rows_of(rng, T, H, "f16")
    logits = rng.normal(size=(T, E)).astype(np.float32)
    logits[:, 4] += 50
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    for k in (1, 2):
        check_moe(dq, x, dev(logits), w1, s1, w2, s2, k, False, "f16", k)
