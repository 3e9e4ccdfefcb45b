"""include/dq4_int8.h without a GPU: its functions are exported, its arguments are checked on the
host before any CUDA call, the binding refuses what does not fit, and the 64-bit definitions that
the GPU tests compare with agree with independent forms of the same."""

import os
import re

import numpy as np
import pytest
import torch

from oracle import int8_layers as defs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 12  # a fake aligned pointer, never followed on these paths
OK, NULL, N_, DTYPE, ALIGN, WORKSPACE = 0, 1, 2, 5, 6, 15


@pytest.fixture(scope="module")
def lib():
    from quantized_weight_dequantization_gb300 import build
    build.build()
    from quantized_weight_dequantization_gb300 import _int8
    return _int8._lib()


def test_declared_functions_are_exported(lib):
    text = open(os.path.join(ROOT, "include", "dq4_int8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*\w+\s+(dq4\w*)\s*\(", text, flags=re.M))
    assert names == {"dq4_int8_quantize", "dq4_int8_quantize_workspace_bytes", "dq4_int8_linear",
                     "dq4_int8_linear_workspace_bytes", "dq4_int8_linear_backward",
                     "dq4_int8_linear_backward_workspace_bytes", "dq4_int8_moe",
                     "dq4_int8_moe_workspace_bytes"}
    for name in names:
        assert hasattr(lib, name)


# ------------------------------------------------------------- refusals, in order
def test_quantize_refusals(lib):
    def call(X=P, stride=64, dt=0, M=4, K=64, thr=6.0, codes=P, scales=P, cols=P, most=8,
             outliers=P, count=P, ws=P, nbytes=1 << 20):
        return lib.dq4_int8_quantize(X, stride, dt, M, K, thr, codes, scales, cols, most, outliers,
                                     count, ws, nbytes, None)
    for kw in ({"M": -1}, {"K": -1}, {"thr": -1.0}, {"thr": float("nan")}, {"most": 0},
               {"most": 129}, {"M": 1 << 31}):
        assert call(**kw) == N_, kw
    assert call(dt=2) == DTYPE and call(dt=3) == DTYPE
    for name in ("X", "codes", "scales", "cols", "outliers", "count"):
        assert call(**{name: None}) == NULL, name
    assert call(M=0, thr=0.0, X=None, codes=None, scales=None) == OK
    for kw in ({"X": P + 1}, {"scales": P + 2}, {"cols": P + 4}, {"outliers": P + 1},
               {"count": P + 2}, {"ws": P + 16}):
        assert call(**kw) == ALIGN, kw
    need = lib.dq4_int8_quantize_workspace_bytes(64)
    assert need > 0 and lib.dq4_int8_quantize_workspace_bytes(-1) == 0
    assert call(ws=None) == WORKSPACE and call(nbytes=need - 1) == WORKSPACE


def test_linear_refusals(lib):
    def call(codes=P, scales=P, CB=P, SCB=P, M=4, N=8, K=64, cols=P, L=2, outliers=P, odt=0,
             bias=P, dt=0, Y=P, ws=P, nbytes=1 << 30, bad=P):
        return lib.dq4_int8_linear(codes, scales, CB, SCB, M, N, K, cols, L, outliers, odt, bias,
                                   dt, Y, ws, nbytes, bad, None)
    for kw in ({"M": -1}, {"N": -1}, {"K": -16}, {"K": 72}, {"L": -1}, {"L": 129}, {"M": 1 << 31},
               {"N": 1 << 31}, {"M": 1 << 30, "K": 1 << 20}):
        assert call(**kw) == N_, kw
    assert call(dt=3) == DTYPE and call(odt=2) == DTYPE and call(odt=2, L=0, M=0) == OK
    assert call(M=0, codes=None, Y=None) == OK and call(N=0, CB=None) == OK
    for name in ("codes", "scales", "CB", "SCB", "cols", "outliers", "Y"):
        assert call(**{name: None}) == NULL, name
    for kw in ({"codes": P + 8}, {"CB": P + 8}, {"scales": P + 2}, {"SCB": P + 2},
               {"cols": P + 4}, {"outliers": P + 1}, {"bias": P + 1}, {"bias": P + 2, "dt": 2},
               {"Y": P + 1}, {"bad": P + 2}):
        assert call(**kw) == ALIGN, kw


def test_backward_refusals(lib):
    def call(dY=P, dt=0, CB=P, SCB=P, M=4, N=8, K=64, dX=P, ws=P, nbytes=1 << 30, bad=P):
        return lib.dq4_int8_linear_backward(dY, dt, CB, SCB, M, N, K, dX, ws, nbytes, bad, None)
    for kw in ({"M": -1}, {"N": -8}, {"K": -16}, {"K": 72}, {"N": 12}, {"M": 1 << 31},
               {"M": 1 << 30, "N": 1 << 20}):
        assert call(**kw) == N_, kw
    assert call(dt=2) == DTYPE
    assert call(M=0, dY=None) == OK and call(K=0, CB=None) == OK
    for name in ("dY", "CB", "SCB", "dX"):
        assert call(**{name: None}) == NULL, name
    for kw in ({"dY": P + 8}, {"CB": P + 8}, {"SCB": P + 2}, {"dX": P + 1}, {"bad": P + 2}):
        assert call(**kw) == ALIGN, kw


def test_moe_refusals(lib):
    need = lib.dq4_int8_moe_workspace_bytes(4, 64, 32, 2)
    assert need > 0
    for shape in ((0, 64, 32, 2), (257, 64, 32, 2), (4, 64, 32, 17), (4, 0, 32, 2)):
        assert lib.dq4_int8_moe_workspace_bytes(*shape) == 0

    def call(X=P, stride=64, dt=0, T=4, H=64, I=32, E=8, logits=P, k=2, w1=P, s1=P, w2=P, s2=P,
             ids=P, weights=P, Y=P, ws=P, nbytes=need, bad=P):
        return lib.dq4_int8_moe(X, stride, dt, T, H, I, E, logits, k, 1, w1, s1, w2, s2, ids,
                                weights, Y, ws, nbytes, bad, None)
    for kw in ({"T": -1}, {"T": 257}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 17, "E": 32},
               {"k": 9}, {"H": 72}, {"I": 40}, {"H": 1 << 16}, {"I": 0},
               {"E": 1024, "H": 1 << 15, "I": 1 << 21}):
        assert call(**kw) == N_, kw
    assert call(dt=2) == DTYPE
    assert call(T=0, X=None) == OK
    for name in ("X", "logits", "w1", "s1", "w2", "s2", "ids", "weights", "Y"):
        assert call(**{name: None}) == NULL, name
    for kw in ({"X": P + 8}, {"stride": 68}, {"logits": P + 2}, {"w1": P + 8}, {"w2": P + 8},
               {"s1": P + 2}, {"s2": P + 2}, {"ids": P + 2}, {"weights": P + 2}, {"Y": P + 1},
               {"ws": P + 16}, {"bad": P + 2}):
        assert call(**kw) == ALIGN, kw
    assert call(ws=None) == WORKSPACE and call(nbytes=need - 1) == WORKSPACE


def test_binding_refuses_host_tensors():
    import quantized_weight_dequantization_gb300 as dq
    x = torch.zeros(4, 64, dtype=torch.float16)
    w, s = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dq.int8_quantize(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dq.int8_linear(dq.Int8Rows(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)), w, s)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dq.int8_linear_backward(torch.zeros(4, 8, dtype=torch.float16), w, s)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dq.int8_moe(x, torch.zeros(4, 2), torch.zeros(2, 64, 64, dtype=torch.int8),
                    torch.zeros(2, 64), torch.zeros(2, 64, 32, dtype=torch.int8),
                    torch.zeros(2, 64), 1)


# ------------------------------------------------------------- the definitions
def test_quantize_definition():
    x = np.array([[1.0, -2.0, 0.5, 8.0], [0, 0, 0, 0], [3.0, np.nan, 1.0, 1.0],
                  [-1.0, 1.0, -7.0, 2.0 ** -110], [2.0 ** -110, 0, 0, 0]])
    codes, scales, cols, outliers, count = defs.quantize(x, 6.0, 3)
    assert cols.tolist() == [2, 3, -1] and count == 2
    assert scales[[0, 1, 3, 4]].tolist() == [2.0, 0.0, 1.0, 0.0] and np.isnan(scales[2])
    assert codes.tolist() == [[64, -127, 0, 0], [0] * 4, [0] * 4, [-127, 127, 0, 0], [0] * 4]
    assert outliers[:, 0].tolist() == [0.5, 0, 1.0, -7.0, 0]
    # columns past the maximum keep codes that end at 127
    codes = defs.quantize(x, 6.0, 1)[0]
    assert codes[0].tolist() == [64, -127, 0, 127] and codes[3, 2] == 0
    # ties go to the even integer
    assert defs.quantize(np.array([[127.0, 0.5, 1.5, -2.5]]))[0].tolist() == [[127, 0, 2, -2]]


def test_linear_definition():
    rng = np.random.default_rng(0)
    codes, CB = (rng.integers(-127, 128, s).astype(np.int8) for s in ((3, 16), (5, 16)))
    scales, SCB = rng.uniform(0.5, 2, 3), rng.uniform(0.5, 2, 5)
    cols, out = np.array([2, 9, 9, 4, -1]), rng.normal(size=(3, 5))
    y, _ = defs.linear(codes, scales, CB, SCB, cols, out)
    for m in range(3):
        for n in range(5):
            want = sum(out[m, 0 if k == 2 else 1] * CB[n, k] * SCB[n] / 127 if k in (2, 9) else
                       int(codes[m, k]) * int(CB[n, k]) * scales[m] * SCB[n] / 127 ** 2
                       for k in range(16))
            assert abs(y[m, n] - want) < 1e-9


def test_linear_backward_is_the_slope_of_the_product():
    rng = np.random.default_rng(1)
    CB, SCB = rng.integers(-127, 128, (6, 16)).astype(np.int8), rng.uniform(0.5, 2, 6)
    x, dy = rng.normal(size=(2, 16)), rng.normal(size=(2, 6))
    w = CB * (SCB[:, None] / 127)
    dx, _ = defs.linear_backward(dy, w)
    step = 1e-5
    for m, k in ((0, 3), (1, 15)):
        a, b = x.copy(), x.copy()
        a[m, k] += step
        b[m, k] -= step
        slope = ((a @ w.T - b @ w.T) * dy).sum() / (2 * step)
        assert abs(slope - dx[m, k]) < 1e-8 * np.abs(w).max() * 100


def test_route_definition():
    inf, nan = np.inf, np.nan
    logits = [[0.0, 1.0, 1.0, -1.0], [-inf] * 4, [nan, 0.0, 2.0, -inf], [-0.0, 0.0, -inf, -inf]]
    ids, weights = defs.route(logits, 2, True)
    assert ids.tolist() == [[1, 2], [0, 1], [2, 1], [0, 1]]
    assert weights[0].tolist() == [0.5, 0.5] and weights[1].tolist() == [0, 0]
    assert np.isnan(weights[2]).all() and weights[3].tolist() == [0.5, 0.5]
    ids, weights = defs.route(logits[:1], 4, False)
    assert abs(weights.sum() - 1) < 1e-12
