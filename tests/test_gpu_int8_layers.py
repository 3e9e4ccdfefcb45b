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


@pytest.mark.parametrize("T", [1, 4, 23, 60])
def test_moe_holds_more_than_its_results(dq, T):
    """FP16 results: the inner values' two terms hold 2^-22 of them, which leaves the results' own
    rounding and FP32 sums."""
    rng = np.random.default_rng(T)
    H, I, E, k = 256, 1424, 8, 2
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    x = rows_of(rng, T, H, "f16")
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    y = dq.int8_moe(x, logits, dev(w1), dev(s1), dev(w2), dev(s2), k)
    want, _, _, size, unit = defs.moe(host(x), host(logits), w1, s1, w2, s2, k, True)
    tol = (unit * (H / 16 * 2.0 ** -23 + 2.0 ** -20)
           + size * (2.0 ** -22 + I / 16 * 2.0 ** -23 + 2.0 ** -19) + U["f16"] * np.abs(want)
           + TINY["f16"])
    close(y, want, tol, T)
    # over all, the rounding of the results is all that is seen: a value's is at most 2^-11 of it
    # and 2^-11 / sqrt(3) in the mean square at most
    off = host(y) - want
    assert np.sqrt((off ** 2).sum() / (want ** 2).sum()) < 2.0 ** -11 / np.sqrt(3)


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


# ------------------------------------------------------------- sums in parts, offsets, ends
@pytest.mark.parametrize("M,N,K", [(40, 64, 65536), (300, 128, 20000), (70, 130, 32768),
                                   (129, 40, 50000), (260, 1500, 8208), (18, 1500, 30000),
                                   (60, 2560, 20480)])
def test_few_tiles_of_long_sums(dq, M, N, K):
    """Few tiles and a long sum: many parts to a tile, of which one joins all; and the same for
    the gradient, twice, bit for bit."""
    rng = np.random.default_rng(M + N + K)
    CB, SCB = weight(rng, N, K)
    rows = random_rows(dq, rng, M, K, 0)
    y = check_linear(dq, rows, CB, SCB, rng.normal(size=N), "f32", (M, N, K))
    assert y.shape == (M, N)
    one, two = (dq.int8_linear(rows, dev(CB), dev(SCB)) for _ in range(2))
    assert torch.equal(one, two)
    lanes = N // 16 * 16
    n = K // 8 * 8
    CB, SCB = weight(rng, n, lanes)
    dy = dev((rng.normal(size=(M, n)) * 0.05).astype(np.float32), DT["f16"])
    dx = dq.int8_linear_backward(dy, dev(CB), dev(SCB))
    w = defs.weight16(CB, SCB, lambda f: f.astype(np.float16).astype(np.float32))
    want, size = defs.linear_backward(host(dy), w)
    close(dx, want, (n / 16 + 4) * 2.0 ** -23 * size + U["f16"] * np.abs(want) + TINY["f16"],
          (M, n, lanes))
    assert torch.equal(dx, dq.int8_linear_backward(dy, dev(CB), dev(SCB)))


@pytest.mark.parametrize("M,N,K", [(40, 1000, 4096), (63, 4001, 2064), (128, 4090, 3000),
                                   (100, 9000, 6160), (250, 4000, 4000), (512, 4000, 8000)])
def test_tiles_shared_by_clusters(dq, M, N, K):
    """Tiles whose sums two, four or eight CTAs share, ragged in every direction."""
    rng = np.random.default_rng(M + N + K)
    K = K // 16 * 16
    CB, SCB = weight(rng, N, K)
    for kind, loud in (("f32", 0), ("bf16", 9)):
        rows = random_rows(dq, rng, M, K, loud)
        check_linear(dq, rows, CB, SCB, rng.normal(size=N), kind, (M, N, K, kind))
        one, two = (dq.int8_linear(rows, dev(CB), dev(SCB)) for _ in range(2))
        assert torch.equal(one, two)
    lanes, n = N // 16 * 16, K // 8 * 8 - 8
    CB, SCB = weight(rng, n, lanes)
    dy = dev((rng.normal(size=(M, n)) * 0.05).astype(np.float32), DT["bf16"])
    w = defs.weight16(CB, SCB, lambda f: torch.from_numpy(f).to(DT["bf16"]).float().numpy())
    want, size = defs.linear_backward(host(dy), w)
    dx = dq.int8_linear_backward(dy, dev(CB), dev(SCB))
    close(dx, want, (n / 16 + 4) * 2.0 ** -23 * size + U["bf16"] * np.abs(want) + TINY["bf16"],
          (M, n, lanes))


@pytest.mark.parametrize("M,N,K", [(64, 4096, 4096), (200, 4096, 2048), (700, 4096, 1024)])
def test_many_rows_in_graphs_on_two_streams(dq, M, N, K):
    """Products of many rows captured twice and replayed on two streams at once, beside eager
    calls on a third, bit for bit what they give alone."""
    rng = np.random.default_rng(M)
    CB, SCB = (dev(a) for a in weight(rng, N, K))
    rows = [random_rows(dq, rng, M, K, 4 * i) for i in range(3)]
    dys = [rows_of(rng, M, N, "bf16") for _ in range(3)]

    def both(i):
        return dq.int8_linear(rows[i], CB, SCB), dq.int8_linear_backward(dys[i], CB, SCB)
    want = [both(i) for i in range(3)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for i in range(2):
            for t in outs[i]:
                t.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            got = both(2)
        torch.cuda.synchronize()
        for a, b in zip((*outs[0], *outs[1], *got), (*want[0], *want[1], *want[2])):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(dq):
    """Operands and results of more than 2^31 values: their last rows, by the definitions."""
    rng = np.random.default_rng(20)
    rows_n, K = 140000, 16384
    x = torch.randn(rows_n, K, device="cuda", dtype=torch.float16,
                    generator=torch.Generator("cuda").manual_seed(1))
    x[rows_n - 1, 7] = 40.0
    rows = dq.int8_quantize(x, 20.0, 4)
    last = slice(rows_n - 40, rows_n)
    codes, scales, *_ = defs.quantize(host(x[last]), 20.0, 4)
    assert rows.cols.tolist() == [7, -1, -1, -1] and rows.count.item() == 1
    assert np.array_equal(rows.codes[last].cpu().numpy(), codes)
    assert np.array_equal(host(rows.scales[last]), scales)
    assert torch.equal(rows.outliers[last, 0], x[last, 7])
    del x

    def check(y, rows, CB, SCB, what):
        want, size = defs.linear(rows.codes.cpu().numpy(), host(rows.scales), CB, SCB,
                                 None if rows.cols is None else rows.cols.cpu().numpy(),
                                 None if rows.cols is None else host(rows.outliers))
        close(y, want, 2.0 ** -21 * size + U["f16"] * np.abs(want) + TINY["f16"], what)
    CB, SCB = weight(rng, 24, K)
    y = dq.int8_linear(rows, dev(CB), dev(SCB))
    cut = dq.Int8Rows(rows.codes[last], rows.scales[last], rows.cols, rows.outliers[last])
    check(y[last], cut, CB, SCB, "rows")
    # the codes as a weight: rows past the 32-bit offset, by few and by many
    few = dq.Int8Rows(dev(rng.integers(-127, 128, (70, K)).astype(np.int8)),
                      dev(np.full(70, 0.7, np.float32)))
    for M in (3, 70):
        some = dq.Int8Rows(few.codes[:M], few.scales[:M])
        y = dq.int8_linear(some, rows.codes, rows.scales)
        check(y[:, last], some, rows.codes[last].cpu().numpy(),
              host(rows.scales[last]).astype(np.float32), M)
    del rows, y, cut
    # results of more than 2^31 values
    M, N, K = 140000, 16400, 16
    CB, SCB = weight(rng, N, K)
    rows = dq.Int8Rows(dev(rng.integers(-127, 128, (M, K)).astype(np.int8)),
                       dev(np.full(M, 0.7, np.float32)))
    y = dq.int8_linear(rows, dev(CB), dev(SCB))
    last = slice(M - 40, M)
    check(y[last], dq.Int8Rows(rows.codes[last], rows.scales[last]), CB, SCB, "results")
    # as dY, and as rows of dX
    dx = dq.int8_linear_backward(y, dev(CB), dev(SCB))
    w = defs.weight16(CB, SCB, lambda f: f.astype(np.float16).astype(np.float32))
    want, size = defs.linear_backward(host(y[last]), w)
    close(dx[last], want, (N / 16 + 4) * 2.0 ** -23 * size + U["f16"] * np.abs(want)
          + TINY["f16"], "dY")
    del y, dx
    CB, SCB = weight(rng, 16, 16400)
    dy = torch.randn(M, 16, device="cuda", dtype=torch.float16)
    dx = dq.int8_linear_backward(dy, dev(CB), dev(SCB))
    w = defs.weight16(CB, SCB, lambda f: f.astype(np.float16).astype(np.float32))
    want, size = defs.linear_backward(host(dy[last]), w)
    close(dx[last], want, 5 * 2.0 ** -23 * size + U["f16"] * np.abs(want) + TINY["f16"], "dX")


@pytest.mark.parametrize("M", [1, 20, 31, 40, 130])
def test_nothing_beside_the_results_is_written(dq, M):
    """Results and workspaces in the middle of larger buffers, at odd sizes."""
    rng = np.random.default_rng(M)
    lib = dq.get_lib()
    N, K, guard = 187, 336, 4096

    def inside(n, dtype):
        buf = torch.full((n + 2 * guard,), 77, dtype=dtype, device="cuda")
        return buf, buf[guard:guard + n]

    def untouched(buf, n, what):
        assert (buf[:guard] == 77).all() and (buf[guard + n:] == 77).all(), what

    def workspace(need):
        buf, ws = inside(need, torch.uint8)
        ws.zero_()
        return buf, ws
    x = rows_of(rng, M, K, "bf16", 7)
    dq.int8_quantize(x)  # (the first call gives the library's functions their types)
    need = lib.dq4_int8_quantize_workspace_bytes(K)
    wb, ws = workspace(need)
    rows = dq.int8_quantize(x, 6.0, 9, workspace=ws)
    untouched(wb, need, "quantize's workspace")
    CB, SCB = weight(rng, N, K)
    for kind in DT:
        need = lib.dq4_int8_linear_workspace_bytes(M, N, K, 9)
        wb, ws = workspace(need)
        yb, y = inside(M * N, DT[kind])
        dq.int8_linear(rows, dev(CB), dev(SCB), Y=y.view(M, N), workspace=ws if need else None)
        untouched(wb, need, (kind, "workspace"))
        untouched(yb, M * N, (kind, "Y"))
        assert torch.equal(y.view(M, N), dq.int8_linear(rows, dev(CB), dev(SCB),
                                                        out_dtype=DT[kind]))
    # (the addresses of 16-bit rows that are odd in units of four bytes)
    yb = torch.full((M * 188 + 1 + guard,), 77, dtype=torch.float16, device="cuda")
    CB, SCB = weight(rng, 188, K)
    dq.int8_linear(rows, dev(CB), dev(SCB), Y=yb[1:1 + M * 188].view(M, 188))
    assert yb[0] == 77 and (yb[1 + M * 188:] == 77).all()
    assert torch.equal(yb[1:1 + M * 188].view(M, 188), dq.int8_linear(rows, dev(CB), dev(SCB)))
    N = 184
    CB, SCB = weight(rng, N, K)
    dy = rows_of(rng, M, N, "bf16")
    need = lib.dq4_int8_linear_backward_workspace_bytes(M, N, K)
    wb, ws = workspace(need)
    xb, dx = inside(M * K, torch.bfloat16)
    dq.int8_linear_backward(dy, dev(CB), dev(SCB), dx.view(M, K), workspace=ws)
    untouched(wb, need, "backward's workspace")
    untouched(xb, M * K, "dX")
    E, H, I = 5, 80, 48
    w1, s1 = weight(rng, E, 2 * I, H)
    w2, s2 = weight(rng, E, H, I)
    need = lib.dq4_int8_moe_workspace_bytes(M, H, I, 2)
    wb, ws = workspace(need)
    args = (rows_of(rng, M, H, "f16"), dev(rng.normal(size=(M, E)).astype(np.float32)), dev(w1),
            dev(s1), dev(w2), dev(s2), 2)
    y = dq.int8_moe(*args, workspace=ws)
    untouched(wb, need, "moe's workspace")
    assert torch.equal(y, dq.int8_moe(*args))


def test_empty(dq):
    """No rows, no outputs, no values."""
    rng = np.random.default_rng(1)
    CB, SCB = weight(rng, 24, 64)
    rows = random_rows(dq, rng, 40, 64, 3)
    none = dq.Int8Rows(rows.codes[:0], rows.scales[:0], rows.cols, rows.outliers[:0])
    assert dq.int8_linear(none, dev(CB), dev(SCB)).shape == (0, 24)
    assert dq.int8_linear(rows, dev(CB[:0]), dev(SCB[:0])).shape == (40, 0)
    for M in (1, 40):
        empty = dq.Int8Rows(rows.codes[:M, :0].contiguous(), rows.scales[:M])
        bias = dev(rng.normal(size=24).astype(np.float32), torch.bfloat16)
        y = dq.int8_linear(empty, dev(CB[:, :0]), dev(SCB), bias, torch.bfloat16)
        assert torch.equal(y, bias.expand(M, -1))
    dy = rows_of(rng, 40, 24, "f16")
    assert dq.int8_linear_backward(dy[:0], dev(CB), dev(SCB)).shape == (0, 64)
    assert dq.int8_linear_backward(dy, dev(CB[:, :0]), dev(SCB)).shape == (40, 0)
    dx = dq.int8_linear_backward(dy[:, :0].contiguous(), dev(CB[:0]), dev(SCB[:0]))
    assert dx.shape == (40, 64) and not dx.any()
    w1, s1 = weight(rng, 2, 32, 48)
    w2, s2 = weight(rng, 2, 48, 16)
    y, ids, p = dq.int8_moe(rows_of(rng, 3, 48, "f16")[:0], torch.empty(0, 2, device="cuda"),
                            dev(w1), dev(s1), dev(w2), dev(s2), 2, return_routing=True)
    assert y.shape == (0, 48) and ids.shape == (0, 2) and p.shape == (0, 2)


# ------------------------------------------------------------- together, and at the same time
def layer(rng, dq, K, N, E=6, I=48):
    w = [dev(a) for a in weight(rng, N, K)]
    up = [dev(a) for a in weight(rng, E, 2 * I, N)]
    down = [dev(a) for a in weight(rng, E, N, I)]
    return w, up, down


def run(dq, x, logits, w, up, down, bias):
    """A projection, a mixture of experts on its result, and the projection's gradient."""
    rows = dq.int8_quantize(x, 6.0, 16)
    y = dq.int8_linear(rows, *w, bias, x.dtype)
    z = dq.int8_moe(y[:8], logits, *up, *down, 2)
    return rows.codes, y, z, dq.int8_linear_backward(y, *w)


@pytest.mark.parametrize("M", [5, 21, 150])
def test_together(dq, M):
    """A layer as it is used, beside the operators that were there: the outlier columns of the
    quantizer through int8_correction_prep, and the 8-bit product by hand."""
    rng = np.random.default_rng(M)
    K, N = 320, 144
    (CB, SCB), up, down = layer(rng, dq, K, N)
    x = rows_of(rng, M, K, "f16", 5)
    bias = dev(rng.normal(size=N).astype(np.float32), torch.float16)
    logits = dev(rng.normal(size=(min(M, 8), 6)).astype(np.float32))
    codes, y, z, dx = run(dq, x, logits, (CB, SCB), up, down, bias)
    rows = dq.int8_quantize(x, 6.0, 16)
    L = rows.count.item()
    assert 0 < L <= 16 and torch.equal(rows.codes, codes)
    cols = rows.cols[:L].contiguous()
    sub_a, sub_b = dq.int8_correction_prep(x, CB, SCB, cols)
    assert torch.equal(sub_a, rows.outliers[:, :L])
    by_hand = (host(codes) @ host(CB).T * host(rows.scales)[:, None] * host(SCB) / 127 ** 2
               + host(sub_a) @ host(sub_b) + host(bias))
    size = (np.abs(host(codes)) @ np.abs(host(CB)).T * host(rows.scales)[:, None] * host(SCB)
            / 127 ** 2 + np.abs(host(sub_a)) @ np.abs(host(sub_b)) + np.abs(host(bias)))
    # (sub_b is the weight in FP16, half a step of which is 2^-11)
    close(y, by_hand, (2.0 ** -21 + 2.0 ** -11) * size + U["f16"] * np.abs(by_hand), M)
    check_moe(dq, y[:8], logits, *(t.cpu().numpy() for t in up), *(t.cpu().numpy() for t in down),
              2, True, "f16", M)
    # the gradient against differences of the product in 64 bits, which is linear in x: along
    # any d, (f(x + d) - f(x - d)) / 2 = <dX, d>.  A weight in FP16 is off by 2^-11 of it.
    dy = y.double()
    W = CB.double() * SCB.double()[:, None] / 127
    f = lambda v: ((v @ W.T) * dy).sum(1)
    for _ in range(4):
        d = torch.randn(M, K, device="cuda", dtype=torch.float64)
        d = d * (torch.rand(M, K, device="cuda") < 0.1)
        want = (f(x.double() + d) - f(x.double() - d)) / 2
        reach = ((dy.abs() @ W.abs()) * d.abs()).sum(1)
        own = (dx.double().abs() * d.abs()).sum(1)
        tol = reach * (2.0 ** -11 + (N / 16 + 4) * 2.0 ** -23) + own * 2.0 ** -11 + 1e-9 * reach
        assert ((dx.double() * d).sum(1) - want).abs().le(tol).all()


def test_gradient_of_codes_against_the_product(dq):
    """The product's own differences: a step of one code moves Y by the column that dX sums."""
    rng = np.random.default_rng(2)
    M, K, N = 37, 64, 48
    CB, SCB = (dev(a) for a in weight(rng, N, K))
    codes = dev(rng.integers(-100, 101, (M, K)).astype(np.int8))
    scales = torch.full((M,), 127.0, device="cuda")  # (a code's step is 1)
    dy = rows_of(rng, M, N, "bf16")
    dx = host(dq.int8_linear_backward(dy, CB, SCB))
    for k in (0, 17, 63):
        hi, lo = codes.clone(), codes.clone()
        hi[:, k] += 16
        lo[:, k] -= 16
        step = (host(dq.int8_linear(dq.Int8Rows(hi, scales), CB, SCB, out_dtype=torch.float32))
                - host(dq.int8_linear(dq.Int8Rows(lo, scales), CB, SCB,
                                      out_dtype=torch.float32))) / 32
        W = np.abs(host(CB) * host(SCB)[:, None] / 127)
        size = np.abs(host(codes)) @ W.T + 16 * W[:, k]
        reach = (np.abs(host(dy)) * size).sum(1)
        # each Y is off by 2^-21 of its magnitudes; the weight in BF16 by 2^-8, dX by 2^-8
        tol = (reach * (2.0 ** -21 + 2.0 ** -24) / 16 + (np.abs(host(dy)) @ W[:, k]) * (2.0 ** -8 + 2.0 ** -19)
               + np.abs(dx[:, k]) * 2.0 ** -8)
        assert (np.abs((host(dy) * step).sum(1) - dx[:, k]) <= tol).all()


@pytest.mark.parametrize("M", [4, 24, 90])
def test_graphs(dq, M):
    """Two captured runs, replayed on two streams at once and in turn with eager calls, give
    what eager calls give."""
    rng = np.random.default_rng(M)
    K, N = 320, 144
    w, up, down = layer(rng, dq, K, N)
    xs = [rows_of(rng, M, K, "bf16", 4) for _ in range(4)]
    logits = [dev(rng.normal(size=(min(M, 8), 6)).astype(np.float32)) for _ in range(4)]
    want = [run(dq, x, l, w, up, down, None) for x, l in zip(xs, logits)]
    torch.cuda.synchronize()
    graphs = []
    for g in range(2):
        x, l = xs[g].clone(), logits[g].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(dq, x, l, w, up, down, None)
        graphs.append((graph, x, l, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(6):
        for g, (graph, x, l, out) in enumerate(graphs):
            at = (turn + g) % 4
            with torch.cuda.stream(streams[g]):
                x.copy_(xs[at])
                l.copy_(logits[at])
        torch.cuda.synchronize()
        for g, (graph, *_) in enumerate(graphs):
            with torch.cuda.stream(streams[g]):
                graph.replay()
        eager = run(dq, xs[3], logits[3], w, up, down, None)
        torch.cuda.synchronize()
        for g, (_, _, _, out) in enumerate(graphs):
            for a, b in zip(out, want[(turn + g) % 4]):
                assert torch.equal(a, b), (turn, g)
        for a, b in zip(eager, want[3]):
            assert torch.equal(a, b), turn


@pytest.mark.parametrize("M", [4, 90])
def test_threads_and_streams(dq, M):
    """Four host threads, two to a stream, and a stream given by its handle."""
    import threading
    rng = np.random.default_rng(M)
    K, N = 320, 144
    w, up, down = layer(rng, dq, K, N)
    xs = [rows_of(rng, M, K, "f16", 4) for _ in range(4)]
    logits = [dev(rng.normal(size=(min(M, 8), 6)).astype(np.float32)) for _ in range(4)]
    want = [run(dq, x, l, w, up, down, None) for x, l in zip(xs, logits)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i % 2]):
                for turn in range(20):
                    at = (i + turn) % 4
                    got = run(dq, xs[at], logits[at], w, up, down, None)
                    streams[i % 2].synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[at])):
                        wrong.append((i, turn))
        except Exception as e:  # noqa: BLE001
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    s = streams[0]
    rows = dq.int8_quantize(xs[0], 6.0, 16, stream=s)
    y = dq.int8_linear(rows, *w, out_dtype=torch.float16, stream=s)
    dx = dq.int8_linear_backward(y, *w, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0][1]) and torch.equal(dx, want[0][3])


def test_repeated_expert_layer(dq):
    """No atomic adds a value: a layer's results are the same each time."""
    rng = np.random.default_rng(12)
    T, H, I, E = 200, 128, 80, 7
    w1, s1 = (dev(a) for a in weight(rng, E, 2 * I, H))
    w2, s2 = (dev(a) for a in weight(rng, E, H, I))
    x = rows_of(rng, T, H, "bf16")
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    y = dq.int8_moe(x, logits, w1, s1, w2, s2, 3)
    for _ in range(5):
        assert torch.equal(y, dq.int8_moe(x, logits, w1, s1, w2, s2, 3))


def test_refused_on_the_device(dq):
    """What only a device's tensors show: shapes, types and strides that are refused before any
    launch."""
    rng = np.random.default_rng(13)
    CB, SCB = (dev(a) for a in weight(rng, 24, 64))
    rows = random_rows(dq, rng, 5, 64, 3)
    E = dq.Dq4Error
    with pytest.raises(E):  # K no multiple of 16
        dq.int8_linear(dq.Int8Rows(rows.codes[:, :40].contiguous(), rows.scales),
                       CB[:, :40].contiguous(), SCB)
    with pytest.raises(E):  # codes off 16 bytes
        off = torch.zeros(5 * 64 + 8, dtype=torch.int8, device="cuda")[8:].view(5, 64)
        dq.int8_linear(dq.Int8Rows(off, rows.scales), CB, SCB)
    with pytest.raises(E):  # a workspace off 256 bytes
        many = random_rows(dq, rng, 60, 64, 0)
        dq.int8_linear(many, CB, SCB,
                       workspace=torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")[16:])
    with pytest.raises(ValueError):
        dq.int8_linear(many, CB, SCB, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    for bad_call in (
            lambda: dq.int8_linear(rows, CB.t(), SCB),
            lambda: dq.int8_linear(rows, CB, SCB[:-1]),
            lambda: dq.int8_linear(rows, CB, SCB, SCB[:-1].half()),
            lambda: dq.int8_linear(rows._replace(cols=None), CB, SCB),
            lambda: dq.int8_linear(rows._replace(outliers=rows.outliers[:, 1:]), CB, SCB),
            lambda: dq.int8_linear(rows, CB, SCB, Y=torch.empty(5, 48, device="cuda")[:, ::2]),
            lambda: dq.int8_quantize(torch.zeros(4, 8, device="cuda").half().t()),
            lambda: dq.int8_quantize(torch.zeros(4, 8, device="cuda").half(), 6.0, 129),
            lambda: dq.int8_linear_backward(torch.zeros(5, 23, device="cuda").half(), CB, SCB)):
        with pytest.raises(ValueError):
            bad_call()
    for bad_call in (lambda: dq.int8_linear(rows, CB.half(), SCB),
                     lambda: dq.int8_linear(rows, CB, SCB, out_dtype=torch.float64),
                     lambda: dq.int8_linear(rows, CB, SCB, SCB),
                     lambda: dq.int8_quantize(torch.zeros(4, 8, device="cuda")),
                     lambda: dq.int8_linear_backward(torch.zeros(5, 24, device="cuda"), CB, SCB)):
        with pytest.raises(TypeError):
            bad_call()
    with pytest.raises(E):  # N no multiple of 8
        dq.int8_linear_backward(torch.zeros(5, 20, device="cuda").half(), CB[:20], SCB[:20])
    w1, s1 = (dev(a) for a in weight(rng, 3, 32, 48))
    w2, s2 = (dev(a) for a in weight(rng, 3, 48, 16))
    x, logits = rows_of(rng, 4, 48, "f16"), torch.zeros(4, 3, device="cuda")
    for bad_call in (lambda: dq.int8_moe(x, logits, w1, s1, w2, s2, 4),
                     lambda: dq.int8_moe(x, logits, w1, s1, w2, s2, 0),
                     lambda: dq.int8_moe(x, logits[:, :2], w1, s1, w2, s2, 2),
                     lambda: dq.int8_moe(x, logits, w1[:, :30], s1, w2, s2, 2),
                     lambda: dq.int8_moe(x[:, :32], logits, w1, s1, w2, s2, 2)):
        with pytest.raises(ValueError):
            bad_call()
    big = torch.zeros(257, 48, device="cuda").half()
    with pytest.raises(E):  # more tokens than the layer is for
        dq.int8_moe(big, torch.zeros(257, 3, device="cuda"), w1, s1, w2, s2, 2)
    # by keyword, every argument
    dq.int8_moe(X=x, logits=logits, w1=w1, s1=s1, w2=w2, s2=s2, top_k=2)
    dq.int8_linear_backward(dY=torch.zeros(5, 24, device="cuda").half(), CB=CB, SCB=SCB)
