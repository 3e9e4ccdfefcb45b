"""Attention over the 8-bit cache where values are no numbers, scores lie far apart, sums are
large, and arguments are at their ends; definitions and tolerances as in test_gpu_attn."""

import sys

import numpy as np
import pytest
import torch

from oracle import attention as oracle_attn
from tests.test_gpu_attn import (DT, MANY, TINY, U, Batch, check_attend, close, dev, dq,  # noqa: F401
                                 host)

pytestmark = pytest.mark.gpu


def both(dq, b, q, new, causal=True, window=0, scale=None, lens=None):
    """(hint, out, lse, bad) of either kernel."""
    cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    lens = dev(np.array(b.lens if lens is None else lens, np.int32))
    for hint in (1, MANY):
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = dq.kv8_attention(b.cache, q, dev(b.table), lens, cu, hint, scale, causal,
                                    window, return_lse=True, bad=bad)
        yield hint, out, lse, int(bad.item())


def definition(b, q, new, scale, causal=True, window=0):
    cu = np.concatenate([[0], np.cumsum(new)])
    with np.errstate(invalid="ignore"):
        return oracle_attn.attend(host(q), b.codes[0], b.codes[1], b.scales[0], b.scales[1],
                                  b.table, b.lens, cu, scale, causal, window)


def tolerance(want, size, reach, dtype):
    """As derived in test_gpu_attn."""
    return ((2.0 ** -10 + 2.0 ** -17 * reach[..., None]) * size + U[dtype] * np.abs(want)
            + TINY[dtype])


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


@pytest.mark.parametrize("dim,heads,kv,page", [(64, 2, 2, 16), (128, 4, 2, 64), (128, 2, 2, 32)])
@pytest.mark.parametrize("lens,new", [([200, 90], [200, 90]), ([200, 90], [102, 8]),
                                      ([167, 90], [6, 3]), ([164, 81], [6, 4])])
def test_attend_rows_before_a_value_that_is_not_finite(dq, dim, heads, kv, page, lens, new):
    """What the append makes of an infinite value of V reaches the rows that see its page; lse
    is as good as out."""
    b = Batch(dq, lens, kv, dim, page, seed=23)

    def make(i, x):
        if i == 1:
            x[min(162, lens[0] - 1), 0, 5] = np.inf  # sequence 0
            x[lens[0] + 80, 1, 0] = np.nan           # sequence 1

    b.append(dq, lens, lens, "bf16", 0, False, make=make)
    assert sum(np.isnan(b.scales[1][t]).sum() for row in b.table for t in row if t >= 0) == 2
    q = dev(b.rng.standard_normal((sum(new), heads, dim)).astype(np.float32), torch.bfloat16)
    want, want_lse, size, reach = definition(b, q, new, dim ** -0.5)
    seen = np.isnan(want).any(-1)
    assert seen.any() and not seen.all()
    for hint, out, lse, bad in both(dq, b, q, new):
        close(host(out), want, tolerance(want, size, reach, "bf16"), ("out", hint))
        close(lse.cpu().numpy()[~seen], want_lse[~seen], 2.0 ** -18 * reach[~seen] + 2.0 ** -18,
              ("lse", hint))
        assert bad == 0


@pytest.mark.parametrize("dim,heads,kv,page", [(64, 2, 2, 16), (128, 8, 2, 64)])
@pytest.mark.parametrize("new", [4, 77])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 50)])
def test_attend_codes_that_are_no_numbers_beside_scales_that_are(dq, dim, heads, kv, page, new,
                                                                 causal, window):
    """A NaN code of a key or a value reaches the rows that see it, and no others."""
    b = Batch(dq, [300, 140], kv, dim, page, seed=24)
    b.fill()
    for i, key, g in ((1, 299, 0), (1, 240, 1), (0, 298, 1), (1, 246, 0)):
        b.codes[i][b.table[0, key // page], g, key % page] = np.nan
    for i, t in ((0, b.cache.k), (1, b.cache.v)):
        t.copy_(dev(b.codes[i].astype(np.float32)).to(torch.float8_e4m3fn))
    q = dev(b.rng.standard_normal((2 * new, heads, dim)).astype(np.float32), torch.bfloat16)
    want, want_lse, size, reach = definition(b, q, [new] * 2, dim ** -0.5, causal, window)
    seen = np.isnan(want).any(-1)
    assert seen.any() and not seen.all()
    for hint, out, lse, _ in both(dq, b, q, [new] * 2, causal, window):
        close(host(out), want, tolerance(want, size, reach, "bf16"), ("out", hint))
        close(lse.cpu().numpy()[~seen], want_lse[~seen], 2.0 ** -18 * reach[~seen] + 2.0 ** -18,
              ("lse", hint))


# ------------------------------------------------------------------ sums and weights
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rise", [0.0, 8.5])
@pytest.mark.parametrize("keys,new", [(20000, 40), (70000, 1)])
def test_attend_many_keys_whose_values_are_zeros(dq, dim, rise, keys, new):
    """All of V at the least scale; the keys after the first 64 score `rise` more: the sum is
    n e^s whatever the scales are.  (Scores are exact, so that lse is good to 2^-18.)"""
    page = 256
    b = Batch(dq, [keys], 1, dim, page, seed=25)
    b.fill()
    for i in range(2):
        b.codes[i] = np.where(np.isnan(b.codes[i]), np.nan, 0.0)
    used = b.table[0, :-(-keys // page)]
    b.codes[0][used, 0, :, 0] = np.where(np.isnan(b.codes[0][used, 0, :, 0]), np.nan, 1.0)
    b.codes[0][b.table[0, 0], 0, :64, 0] = 0.0
    b.scales[0][used], b.scales[1][used] = 1.0, 2.0 ** -100
    for i, (t, s) in enumerate(((b.cache.k, b.cache.k_scale), (b.cache.v, b.cache.v_scale))):
        t.copy_(dev(b.codes[i].astype(np.float32)).to(torch.float8_e4m3fn))
        s.copy_(dev(b.scales[i]))
    q = torch.zeros((new, 4, dim), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = rise
    seen = np.arange(keys - new, keys) + 1
    want = np.log(64 + (seen - 64) * np.exp(rise))[:, None].repeat(4, 1)
    for hint, out, lse, bad in both(dq, b, q, [new], scale=1.0):
        assert not bool(out.any()), hint
        close(lse.cpu().numpy(), want, 2.0 ** -18 * rise + 2.0 ** -18 * np.abs(want), hint)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("v_exp", [-100, 0, 110])
def test_attend_values_at_the_ends_of_the_scales(dq, dim, v_exp):
    """V at the least scale that append writes, and near the largest; BF16 holds the results."""
    b = Batch(dq, [3000, 65], 2, dim, 64, seed=26)
    b.fill()
    b.scales[1] = np.where(np.isnan(b.scales[1]), np.nan, 2.0 ** v_exp).astype(np.float32)
    b.cache.v_scale.copy_(dev(b.scales[1]))
    check_attend(dq, b, [1, 1], 4, "bf16")
    check_attend(dq, b, [130, 40], 4, "bf16")


@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 32)])
@pytest.mark.parametrize("above", [0, 3])
def test_attend_values_beside_one_dominant_key_of_zeros(dq, dim, heads, above):
    """The first key scores 12 to 17 nats above the others and has no values, so that the result
    is what the small weights give (`above`: some later keys pass the first one by 1.5 nats, with
    no values either).  The others' scores are equal: their roundings do not average out."""
    n, page, kv = 700, 64, 2
    b = Batch(dq, [n], kv, dim, page, seed=27)
    b.fill()
    for i in range(2):
        b.codes[i] = np.where(np.isnan(b.codes[i]), np.nan, np.abs(b.codes[i]))
    for t in b.table[0]:
        b.scales[0][t], b.scales[1][t] = 1.0, 256.0
        b.codes[0][t] = np.where(np.isnan(b.codes[0][t]), np.nan, 0.0)
    for key, code in [(0, 1.0)] + [(100 + 70 * i, 1.125) for i in range(above)]:
        b.codes[0][b.table[0, key // page], :, key % page, 0] = code
        b.codes[1][b.table[0, key // page], :, key % page] = 0.0
    for i, (t, s) in enumerate(((b.cache.k, b.cache.k_scale), (b.cache.v, b.cache.v_scale))):
        t.copy_(dev(b.codes[i].astype(np.float32)).to(torch.float8_e4m3fn))
        s.copy_(dev(b.scales[i]))
    new = 150
    q = np.zeros((new, heads, dim), np.float32)
    q[:, :, 0] = np.linspace(12, 17, new * heads).reshape(new, heads)
    q = dev(q, torch.float16)
    want, want_lse, size, reach = definition(b, q, [new], 1.0)
    for hint, out, lse, bad in both(dq, b, q, [new], scale=1.0):
        close(host(out), want, tolerance(want, size, reach, "f16"), ("out", hint))
        close(lse.cpu().numpy(), want_lse, 2.0 ** -18 * reach + 2.0 ** -18, ("lse", hint))


# ---------------------------------------------------------------- uneven sequences
@pytest.mark.parametrize("dim,heads,kv", [(128, 4, 1), (64, 4, 2)])
def test_attend_sequences_of_one_tile_after_sequences_of_two(dq, dim, heads, kv):
    """Long chunks that many CTAs share, then prompts of two tiles and a step or two, then single
    tokens, which have no rows in the second tile: it must not fall behind the first by more
    steps than scales are kept for."""
    lens, new = [], []
    for i in range(6):
        lens += [6000 + 300 * i, 40, 90] + [500 + 90 * i] * 4
        new += [130, 40, 70] + [1] * 4
    b = Batch(dq, lens, kv, dim, 64, seed=30)
    b.fill()
    first = check_attend(dq, b, new, heads, "bf16", max_new=MANY)
    b.rng = np.random.default_rng(31)
    state = b.rng.bit_generator.state
    for _ in range(3):
        b.rng.bit_generator.state = state
        again = check_attend(dq, b, new, heads, "bf16", max_new=MANY)
        assert torch.equal(again[0], again[2]) and len(first) == 3


# --------------------------------------------------------------------- captured calls
def captured(fn, stream=None):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = fn()
    return graph, out


@pytest.mark.parametrize("hint", [1, MANY])
def test_attend_and_norm_backward_captured_without_a_call_before(dq, hint):
    """On the capture's own stream, which no call has used."""
    b = Batch(dq, [700, 90], 2, 128, 64, seed=32)
    b.fill()
    q = dev(b.rng.standard_normal((60, 4, 128)).astype(np.float32), torch.bfloat16)
    cu = dev(np.array([0, 30, 60], np.int32))
    args = (b.cache, q, dev(b.table), dev(np.array(b.lens, np.int32)), cu, hint)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    norm = (q, q, q, q, w, w)
    want, grads = dq.kv8_attention(*args), dq.qk_norm_rope_backward(*norm)
    side = torch.cuda.Stream()
    for stream in (None, side):
        graph, out = captured(lambda: (dq.kv8_attention(*args), dq.kv8_attention(*args),
                                       *dq.qk_norm_rope_backward(*norm)), stream)
        for _ in range(3):
            for o in out:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want) and torch.equal(out[1], want)
            assert all(torch.equal(x, y) for x, y in zip(out[2:], grads))


@pytest.mark.parametrize("hint", [1, MANY])
def test_captured_calls_share_no_workspace(dq, hint):
    """Two graphs captured on one stream, replayed side by side with calls of other shapes."""
    b = Batch(dq, [9000, 90, 4000], 2, 64, 64, seed=33)
    b.fill()
    table, lens = dev(b.table), dev(np.array(b.lens, np.int32))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    calls = []
    for new in (40, 25, 60):
        q = dev(b.rng.standard_normal((3 * new, 4, 64)).astype(np.float32), torch.bfloat16)
        cu = dev(np.arange(4, dtype=np.int32) * new)
        calls.append(lambda q=q, cu=cu: (dq.kv8_attention(b.cache, q, table, lens, cu, hint),
                                         *dq.qk_norm_rope_backward(q, q, q, q, w, w)))
    want = [call() for call in calls]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls[2]()  # the stream has a workspace of its own
    torch.cuda.synchronize()
    graphs = [captured(call, side) for call in calls[:2]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(side):
            eager = calls[2]()
        torch.cuda.synchronize()
        for got, expected in zip([g[1] for g in graphs] + [eager], want):
            assert all(torch.equal(x, y) for x, y in zip(got, expected))


# ---------------------------------------------------------------- ends of arguments
@pytest.mark.parametrize("dim", [64, 72])
def test_tables_without_rows_have_no_position(dq, dim):
    """Tables of no rows are not "no tables": every position is outside them."""
    x = torch.randn((3, 2, dim), device="cuda").bfloat16()
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    t = torch.empty((0, dim // 2), device="cuda")
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = dq.qk_norm_rope(x, x, w, w, t, t, pos, bad=bad)
    assert not bool(q.any()) and not bool(k.any()) and int(bad.item()) == 12
    bad.zero_()
    grads = dq.qk_norm_rope_backward(x, x, x, x, w, w, t, t, pos, bad=bad)
    assert not any(bool(g.any()) for g in grads) and int(bad.item()) == 12


def test_append_tables_without_rows_store_zeros(dq):
    b = Batch(dq, [3], 2, 64, 16, seed=28)
    x = torch.randn((3, 2, 64), device="cuda").bfloat16()
    t = torch.empty((0, 32), device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    dq.kv8_append(b.cache, x, x, dev(b.table), dev(np.array([3], np.int32)),
                  dev(np.array([0, 3], np.int32)), t, t, bad=bad)
    at = int(b.table[0, 0])
    assert int(bad.item()) == 3 and not bool(b.cache.k[at, :, :3].float().any())
    assert bool(b.cache.v[at, :, :3].float().any())


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, sys.maxsize])
def test_attend_windows_longer_than_any_sequence(dq, window):
    b = Batch(dq, [300, 140, 3], 2, 64, 16, seed=29)
    b.fill()
    q = dev(b.rng.standard_normal((45, 4, 64)).astype(np.float32), torch.bfloat16)
    cu = dev(np.array([0, 20, 40, 45], np.int32))  # (two rows lie before sequence 2's start)
    args = (b.cache, q, dev(b.table), dev(np.array(b.lens, np.int32)), cu)
    for hint in (1, MANY, 2 ** 31, 2 ** 40):
        for causal in (True, False):
            assert torch.equal(dq.kv8_attention(*args, hint, causal=causal, window=window),
                               dq.kv8_attention(*args, hint, causal=causal))
