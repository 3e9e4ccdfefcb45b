"""Norm with rotation, the 8-bit cache's append and the attention over it, on the GPU against
the 64-bit definitions of oracle/attention.py.

Tolerances, from the arithmetic.  u is half a step of the output type relative to its value.
 * norm: FP32 sums of up to 1024 squares (37 additions deep), a square root and at most five
   roundings: 2^-18 of the magnitudes that meet in a value, plus u |y|.
 * its gradients: the same, twice over: 2^-17; weight gradients: sums at most a few hundred
   additions deep: 2^-15 of the summed magnitudes.
 * append: bit for bit (the rotation is defined in FP32, scales are powers of two).
 * attention: scores from exact 16-bit operands with FP32 sums, 2^-18 of the magnitudes (delta);
   weights rounded to FP16: 2^-10 with their normalization; so (2^-10 + 2 delta) sum p |v| plus
   u |out|.  lse: delta + 2^-18.
"""

import numpy as np
import pytest
import torch

from oracle import attention as oracle_attn

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
    return t.detach().float().cpu().numpy()


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), what
    over = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    assert not over.size or over.max() <= 0, (what, float(over.max()), int((over > 0).sum()))


def tables(rows, rotary, rng):
    angle = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rotary, 2) / rotary)
    angle = angle + rng.uniform(0, 6, angle.shape)
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


# ------------------------------------------------------------------ norm and rotation
NORM = [
    # tokens, heads, kv heads, dim, rotary, dtype, interleaved
    (1, 1, 1, 64, 64, "bf16", False), (1, 32, 8, 128, 128, "bf16", False),
    (5, 7, 3, 64, 32, "f16", True), (33, 9, 1, 256, 256, "bf16", False),
    (67, 4, 2, 128, 72, "f32", False), (130, 5, 5, 128, 8, "f16", False),
    (700, 32, 8, 128, 128, "f16", True), (3, 2, 1, 80, 80, "bf16", False),
    (17, 3, 1, 96, 30, "f32", True), (9, 2, 2, 2, 2, "f16", False),
    (4, 1, 1, 1024, 500, "bf16", False), (6, 3, 2, 128, 12, "bf16", True),
    (1500, 40, 8, 64, 64, "bf16", False), (2, 3, 0, 128, 128, "bf16", False),
    (0, 4, 2, 128, 128, "bf16", False),
]


def norm_problem(tokens, heads, kv, dim, rotary, dtype, seed, pad=0):
    rng = np.random.default_rng(seed)
    fused = dev(rng.standard_normal((tokens, heads + 2 * kv + 1, dim + pad)).astype(np.float32),
                DT[dtype])
    q = fused[:, :heads, :dim]
    k = fused[:, heads:heads + kv, :dim] if kv else None
    weights = [dev((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32), DT[dtype])
               for _ in range(2)]
    cos, sin = tables(97, rotary, rng)
    return q, k, weights, cos, sin, rng.integers(0, 97, tokens), rng


def check_norm(dq, q, k, weights, cos, sin, positions, dtype, interleaved, outs, eps=1e-5):
    for x, w, y in zip((q, k), weights, outs):
        if x is None:
            assert y is None
            continue
        want, size = oracle_attn.norm_rope(host(x), None if w is None else host(w), cos, sin,
                                           positions, eps, interleaved)
        assert y.is_contiguous() and y.dtype == x.dtype
        close(host(y), want, 2.0 ** -18 * size + U[dtype] * np.abs(want) + TINY[dtype], "norm")


@pytest.mark.parametrize("case", NORM, ids=str)
@pytest.mark.parametrize("pad", [0, 4, 3])
def test_norm_forward_and_backward(dq, case, pad):
    tokens, heads, kv, dim, rotary, dtype, inter = case
    q, k, w, cos, sin, pos, rng = norm_problem(tokens, heads, kv, dim, rotary, dtype, 1, pad)
    args = (q, k, w[0], w[1] if kv else None, dev(cos), dev(sin), dev(pos), 1e-5, inter)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = dq.qk_norm_rope(*args, bad=bad)
    check_norm(dq, q, k, w, cos, sin, pos, dtype, inter, outs)
    grads = [None if x is None else dev(rng.standard_normal(x.shape).astype(np.float32),
                                        DT[dtype]) for x in (q, k)]
    got = dq.qk_norm_rope_backward(*grads, *args, bad=bad)
    again = dq.qk_norm_rope_backward(*grads, *args)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    for i, (x, dy) in enumerate(zip((q, k), grads)):
        if x is None:
            assert got[i] is None and got[2 + i] is None
            continue
        dx, dx_size, dw, dw_size = oracle_attn.norm_rope_backward(
            host(dy), host(x), host(w[i]), cos, sin, pos, 1e-5, inter)
        close(host(got[i]), dx, 2.0 ** -17 * dx_size + U[dtype] * np.abs(dx) + TINY[dtype], "dx")
        assert got[2 + i].dtype == torch.float32
        close(host(got[2 + i]), dw, 2.0 ** -15 * dw_size + 1e-30, "dw")
    assert int(bad.item()) == 0


@pytest.mark.parametrize("dim", [64, 80, 128])
def test_norm_alone_and_rotation_alone(dq, dim):
    q, k, w, cos, sin, pos, rng = norm_problem(19, 5, 2, dim, dim // 2, "f16", 2)
    outs = dq.qk_norm_rope(q, k, w[0], w[1], eps=1e-5)
    check_norm(dq, q, k, w, None, None, None, "f16", False, outs)
    outs = dq.qk_norm_rope(q, k, None, None, dev(cos), dev(sin), dev(pos))
    check_norm(dq, q, k, (None, None), cos, sin, pos, "f16", False, outs)
    dy = dev(rng.standard_normal(q.shape).astype(np.float32), torch.float16)
    dx, _, dw, _ = dq.qk_norm_rope_backward(dy, None, q, None, None, None, dev(cos), dev(sin),
                                            dev(pos))
    assert dw is None
    want, size, _, _ = oracle_attn.norm_rope_backward(host(dy), host(q), None, cos, sin, pos,
                                                      1e-5, False)
    close(host(dx), want, 2.0 ** -18 * size + U["f16"] * np.abs(want) + TINY["f16"], "turned")


@pytest.mark.parametrize("dim", [64, 48])
def test_norm_gradient_against_differences(dq, dim):
    """(f(x + h e) - f(x - h e)) / 2h of the loss sum(y * dy), in float64 on the definition, and
    the kernel's gradients in float32."""
    q, _, w, cos, sin, pos, rng = norm_problem(2, 2, 0, dim, 16, "f32", 3)
    dy = rng.standard_normal(q.shape)
    dx, _, dw, _ = dq.qk_norm_rope_backward(dev(dy.astype(np.float32)), None, q, None, w[0], None,
                                            dev(cos), dev(sin), dev(pos), 1e-5)
    x64, w64 = host(q).astype(np.float64), host(w[0]).astype(np.float64)
    dy64 = dy.astype(np.float32).astype(np.float64)

    def loss(x, weight):
        return float((oracle_attn.norm_rope(x, weight, cos, sin, pos, 1e-5, False)[0]
                      * dy64).sum())

    h = 1e-6  # differences are good to about h^2 + 1e-16 |loss| / h, 1e-8 here
    for at in [(0, 0, 0), (0, 1, 5), (1, 0, dim - 1), (1, 1, 17)]:
        step = np.zeros_like(x64)
        step[at] = h
        slope = (loss(x64 + step, w64) - loss(x64 - step, w64)) / (2 * h)
        assert abs(float(dx[at]) - slope) <= 2e-5 * max(1.0, abs(slope))
    for i in (0, 7, dim - 1):
        step = np.zeros_like(w64)
        step[i] = h
        slope = (loss(x64, w64 + step) - loss(x64, w64 - step)) / (2 * h)
        assert abs(float(dw[i]) - slope) <= 2e-5 * max(1.0, abs(slope))


@pytest.mark.parametrize("dim", [128, 72])
def test_norm_positions_outside_the_tables_give_zeros_and_are_counted(dq, dim):
    q, k, w, cos, sin, pos, rng = norm_problem(6, 3, 2, dim, 16, "bf16", 4)
    pos[[1, 4]] = [-1, 97]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = dq.qk_norm_rope(q, k, w[0], w[1], dev(cos), dev(sin), dev(pos), bad=bad)
    assert int(bad.item()) == 2 * 5
    keep = [0, 2, 3, 5]
    for y in (a, b):
        assert not y[[1, 4]].any() and y[keep].any(-1).all()
    grads = [torch.ones_like(y) for y in (a, b)]
    got = dq.qk_norm_rope_backward(*grads, q, k, w[0], w[1], dev(cos), dev(sin), dev(pos))
    rest = dq.qk_norm_rope_backward(*[g[keep].contiguous() for g in grads], q[keep], k[keep],
                                    w[0], w[1], dev(cos), dev(sin), dev(pos[keep]))
    assert not got[0][[1, 4]].any() and torch.equal(got[0][keep], rest[0])
    for x, y in zip(got[2:], rest[2:]):
        torch.testing.assert_close(x, y, rtol=1e-5, atol=1e-5)


def guarded(need):
    """A zero-filled workspace of just `need` bytes, and the bytes that follow it."""
    buf = torch.zeros(need + 65536, dtype=torch.uint8, device="cuda")
    buf[need:] = 0xA5
    return buf[:need], buf[need:]


@pytest.mark.parametrize("dim,pad", [(128, 0), (64, 3), (80, 0), (256, 3)])
def test_norm_backward_stays_in_its_workspace(dq, dim, pad):
    """As many CTAs as there can be leave sums: pad 3 and dim 80 take the any-size kernel."""
    from quantized_weight_dequantization_gb300 import _attention
    q, k, w, cos, sin, pos, rng = norm_problem(900, 6, 3, dim, 64, "bf16", 4, pad)
    grads = [dev(rng.standard_normal(x.shape).astype(np.float32), torch.bfloat16) for x in (q, k)]
    ws, after = guarded(_attention._norm_need(dim))
    got = dq.qk_norm_rope_backward(*grads, q, k, *w, dev(cos), dev(sin), dev(pos), 1e-5,
                                   workspace=ws)
    assert bool((after == 0xA5).all()) and not bool(ws[:256].any())
    for i, (x, dy) in enumerate(zip((q, k), grads)):
        _, _, dw, dw_size = oracle_attn.norm_rope_backward(host(dy), host(x), host(w[i]), cos, sin,
                                                           pos, 1e-5, False)
        close(host(got[2 + i]), dw, 2.0 ** -15 * dw_size + 1e-30, "dw")


# ----------------------------------------------------------------------- the cache
class Batch:
    """A ragged batch on pages in random order, slots and scales never written left as NaN."""

    def __init__(self, dq, lens, kv_heads, dim, page, seed, extra_width=0):
        self.rng = np.random.default_rng(seed)
        self.lens, self.page, self.dim, self.kv = list(lens), page, dim, kv_heads
        held = [-(-n // page) for n in lens]
        self.pages = sum(held) + 2
        order = self.rng.permutation(self.pages)
        width = max(1, max(held, default=1)) + extra_width
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, kv_heads, page, dim)
        self.cache = dq.KV8Cache.empty(self.pages, kv_heads, page, dim)
        self.codes, self.scales = [], []
        for codes, scales in ((self.cache.k, self.cache.k_scale),
                              (self.cache.v, self.cache.v_scale)):
            codes.view(torch.uint8).fill_(0x7F)
            scales.fill_(float("nan"))
            self.codes.append(np.full(shape, np.nan))
            self.scales.append(np.full(shape[:2], np.nan, np.float32))

    def fill(self, spread=1.0):
        """Random codes and scales wherever a sequence has tokens."""
        for i, (codes, scales) in enumerate(((self.cache.k, self.cache.k_scale),
                                             (self.cache.v, self.cache.v_scale))):
            for b, n in enumerate(self.lens):
                for j in range(-(-n // self.page)):
                    at = self.table[b, j]
                    m = min(self.page, n - j * self.page)
                    self.codes[i][at, :, :m] = oracle_attn.e4m3(
                        np.clip(60 * self.rng.standard_normal((self.kv, m, self.dim)), -448, 448))
                    self.scales[i][at] = 2.0 ** np.round(
                        -6 + spread * self.rng.standard_normal(self.kv))
            codes.copy_(dev(self.codes[i].astype(np.float32)).to(torch.float8_e4m3fn))
            scales.copy_(dev(self.scales[i]))

    def check(self):
        for i, (codes, scales) in enumerate(((self.cache.k, self.cache.k_scale),
                                             (self.cache.v, self.cache.v_scale))):
            assert np.array_equal(scales.cpu().numpy(), self.scales[i], equal_nan=True)
            got, want = host(codes), self.codes[i]
            assert np.array_equal(np.isnan(got), np.isnan(want))
            assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])

    def append(self, dq, new, lens, dtype, rotary, inter, use_cu=True, make=None, strided=False):
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        tokens = int(cu[-1])
        xs = []
        for i in range(2):
            x = self.rng.standard_normal((tokens, self.kv, self.dim)).astype(np.float32)
            x *= np.exp(self.rng.standard_normal((tokens, 1, 1)))
            if make:
                make(i, x)
            xs.append(dev(x, DT[dtype]))
        if strided:
            fused = torch.stack(xs, 1).contiguous()  # tokens x 2 x heads x dim
            xs = [fused[:, 0], fused[:, 1]]
        cos = sin = None
        if rotary:
            cos, sin = tables(max(max(lens), 1) + 3, rotary, self.rng)
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        dq.kv8_append(self.cache, xs[0], xs[1], dev(self.table), dev(np.array(lens, np.int32)),
                      dev(cu) if use_cu else None, None if cos is None else dev(cos),
                      None if sin is None else dev(sin), inter, bad=bad)
        for i in range(2):
            oracle_attn.append(self.codes[i], self.scales[i], host(xs[i]),
                               cos if i == 0 else None, sin, self.table, lens, cu, inter)
        assert int(bad.item()) == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim,dtype,rotary,inter", [
    (128, "bf16", 128, False), (64, "f16", 64, True), (128, "f16", 72, False),
    (64, "bf16", 8, True), (64, "bf16", 0, False)])
def test_append_prompts_then_tokens(dq, page, dim, dtype, rotary, inter):
    """A prompt for each sequence, then two ragged steps and three of single tokens."""
    final = [1, 17, page, page + 1, 3 * page + 9, 700, 5]
    b = Batch(dq, [n + 8 for n in final], 3, dim, page, seed=page + dim)
    lens = list(final)
    b.append(dq, final, lens, dtype, rotary, inter)
    b.check()
    for new in ([0, 1, 2, 0, 3, 1, 0], [2, 0, 1, 1, 0, 3, 2]):
        lens = [n + m for n, m in zip(lens, new)]
        b.append(dq, new, lens, dtype, rotary, inter, strided=True)
    for _ in range(3):
        lens = [n + 1 for n in lens]
        b.append(dq, [1] * len(lens), lens, dtype, rotary, inter, use_cu=False)
    b.check()


@pytest.mark.parametrize("pad", [4, 8])
@pytest.mark.parametrize("dim,rotary,inter", [(128, 128, False), (64, 32, True), (64, 8, False)])
def test_append_tokens_aligned_to_8_or_16_bytes(dq, pad, dim, rotary, inter):
    """Rows a multiple of 4 or of 8 values apart, the first 8 bytes past a 16-byte boundary."""
    b = Batch(dq, [100, 37], 3, dim, 32, seed=16)
    buf = b.rng.standard_normal((2, 137, 3, dim + pad)).astype(np.float32)
    flat = [torch.zeros(buf[0].size + 8, dtype=torch.bfloat16, device="cuda")[4:-4]
            for _ in range(2)]
    xs = []
    for t, x in zip(flat, buf):
        t.copy_(dev(x.ravel(), torch.bfloat16))
        xs.append(t.view(137, 3, dim + pad)[:, :, :dim])
    cos, sin = tables(101, rotary, b.rng)
    lens, cu = np.array([100, 37], np.int32), np.array([0, 100, 137], np.int32)
    dq.kv8_append(b.cache, *xs, dev(b.table), dev(lens), dev(cu), dev(cos), dev(sin), inter)
    for i in range(2):
        oracle_attn.append(b.codes[i], b.scales[i], host(xs[i]), cos if i == 0 else None, sin,
                           b.table, lens, cu, inter)
    b.check()


def test_append_scales_grow_shrink_and_hit_their_limits(dq):
    b = Batch(dq, [64] * 6, 2, 64, 64, seed=9)
    sizes = [1.0, 448.0, 449.0, 1e-38, 6e4, 0.0]

    def put(level):
        def make(i, x):
            x[:] = np.clip(x, -1, 1)
            x[:, :, 0] = 1.0
            x *= np.array(sizes)[:, None, None].astype(np.float32) * np.float32(level)
        return make

    for step, level in enumerate((1.0, 0.25, 3.0, 2.0 ** -9, 100.0)):
        b.append(dq, [1] * 6, [step + 1] * 6, "bf16", 0, False, use_cu=False, make=put(level))
        b.check()


def test_append_values_that_are_not_finite_mark_their_page_and_head_alone(dq):
    b = Batch(dq, [40, 40], 2, 128, 16, seed=10)

    def make(i, x):
        x[3, 0, 5] = np.nan
        x[21, 1, 127] = np.inf
        x[45, 0, 0] = -np.inf

    b.append(dq, [34, 34], [34, 34], "f16", 64, False, make=make)
    assert sum(np.isnan(s[t]).sum() for s in b.scales for t in b.table[:, :2].ravel()) == 6
    b.append(dq, [6, 6], [40, 40], "f16", 64, False)
    b.check()


def test_append_counts_tokens_without_a_place(dq):
    b = Batch(dq, [40, 20, 33], 2, 64, 16, seed=11)
    b.table[0, 1] = b.pages  # no such page: tokens 16 .. 31 of sequence 0
    before = [t.clone() for t in (b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8))]
    x = dev(b.rng.standard_normal((93, 2, 64)).astype(np.float32), torch.bfloat16)
    cos, sin = tables(36, 64, b.rng)  # keys 36 .. 39 of sequence 0 are past the tables
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    dq.kv8_append(b.cache, x, x, dev(b.table[:, :3]), dev(np.array([40, 17, 33], np.int32)),
                  dev(np.array([0, 40, 60, 93], np.int32)), dev(cos), dev(sin), bad=bad)
    # sequence 1 has 20 tokens for a length of 17: positions -3 .. 16
    assert int(bad.item()) == 16 + 3 + 4
    assert not b.cache.k[int(b.table[0, 2])][:, 4:8].float().any()
    used = set(int(t) for t in b.table[0, [0, 2]]) | set(int(t) for t in b.table[1, :2]) | set(
        int(t) for t in b.table[2, :3])
    idle = [i for i in range(b.pages) if i not in used]
    for was, now in zip(before, (b.cache.k, b.cache.v)):
        assert torch.equal(was[idle], now.view(torch.uint8)[idle])


# ------------------------------------------------------------------------ attention
MANY = 1 << 20  # as max_new: the kernel for many rows, whatever the sizes; 1: the one for few


def check_attend(dq, b, new, heads, dtype, causal=True, window=0, scale=None, max_new=None,
                 use_cu=True, q_scale=1.0, strided=False, lens=None, stream=None):
    """Both kernels, and the one that the call would choose, against the definition; returns the
    outputs."""
    lens = b.lens if lens is None else lens
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    x = b.rng.standard_normal((int(cu[-1]), heads, b.dim)).astype(np.float32) * q_scale
    q = dev(x, DT[dtype])
    if strided:
        q = torch.cat([q, q[:, :1], q[:, :1]], 1)[:, :heads]
    scale = b.dim ** -0.5 if scale is None else scale
    want, want_lse, size, reach = oracle_attn.attend(
        host(q), b.codes[0], b.codes[1], b.scales[0], b.scales[1], b.table, lens, cu, scale,
        causal, window)
    if dtype == "f16":  # past the type's range an output is infinite
        want = np.where(np.abs(want) < 65520, want, np.copysign(np.inf, want))
    delta = 2.0 ** -18 * reach
    outs = []
    for hint in (max_new, 1, MANY):
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = dq.kv8_attention(b.cache, q, dev(b.table), dev(np.array(lens, np.int32)),
                                    dev(cu) if use_cu else None, hint, scale, causal, window,
                                    return_lse=True, bad=bad, stream=stream)
        if stream is not None:
            stream.synchronize()
        close(host(out), want, (2.0 ** -10 + 2 * delta[..., None]) * size
              + U[dtype] * np.abs(want) + TINY[dtype], ("out", hint))
        close(lse.cpu().numpy(), want_lse, delta + 2.0 ** -18, ("lse", hint))
        assert int(bad.item()) == 0
        outs.append(out)
    return outs


LENS = [1, 0, 15, 16, 31, 33, 64, 65, 127, 300, 2]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim,heads,kv,dtype", [
    (128, 32, 8, "bf16"), (64, 6, 2, "f16"), (128, 3, 3, "f16"), (64, 16, 1, "bf16"),
    (128, 40, 1, "bf16"), (64, 35, 5, "bf16")])
def test_attend_single_tokens(dq, page, dim, heads, kv, dtype):
    b = Batch(dq, LENS, kv, dim, page, seed=page + heads, extra_width=3)
    b.fill()
    check_attend(dq, b, [1] * len(LENS), heads, dtype, use_cu=False)


@pytest.mark.parametrize("window", [0, 1, 7, 64, 129])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 128)])
def test_attend_several_tokens(dq, window, causal, dim, page):
    """Few new tokens a sequence, none for some; a row before the sequence's start is empty."""
    b = Batch(dq, LENS, 2, dim, page, seed=window + page)
    b.fill()
    check_attend(dq, b, [1, 0, 3, 4, 5, 2, 1, 4, 6, 3, 2], 4, "bf16", causal, window, max_new=6)
    check_attend(dq, b, [1, 2, 3, 4, 5, 2, 1, 4, 6, 3, 7], 6, "f16", causal, window, max_new=2)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,heads,kv,page,dtype", [
    (128, 8, 2, 64, "bf16"), (64, 4, 4, 16, "f16"), (128, 5, 1, 256, "f16"),
    (64, 21, 3, 32, "bf16")])
def test_attend_prompts(dq, window, causal, dim, heads, kv, page, dtype):
    b = Batch(dq, [300, 129, 1, 0, 77, 520], kv, dim, page, seed=heads)
    b.fill()
    check_attend(dq, b, [300, 129, 1, 0, 70, 33], heads, dtype, causal, window, max_new=300)
    check_attend(dq, b, [128, 1, 1, 3, 64, 257], heads, dtype, causal, window, strided=True)


def test_attend_long_sequence(dq):
    b = Batch(dq, [9001, 20], 1, 64, 128, seed=5)
    b.fill()
    check_attend(dq, b, [1, 1], 4, "bf16", use_cu=False)
    check_attend(dq, b, [2, 9], 2, "f16", window=5000)
    check_attend(dq, b, [60, 20], 4, "bf16")


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend_scales_far_apart_and_sharp_scores(dq, new, dtype):
    """Pages whose scales differ by 2^40, and scores that leave one key nearly alone."""
    b = Batch(dq, [700, 130], 2, 128, 16, seed=6)
    b.fill(spread=6.0)
    b.scales[0][:] = np.where(np.isnan(b.scales[0]), np.nan, 2.0 ** -6)
    b.cache.k_scale.copy_(dev(b.scales[0]))
    check_attend(dq, b, [new, new], 4, dtype, q_scale=8.0)
    check_attend(dq, b, [new, new], 4, dtype, q_scale=2.0 ** -12, scale=1.0)
    check_attend(dq, b, [new, new], 4, dtype, scale=0.0)
    check_attend(dq, b, [new, new], 4, dtype, scale=-0.1)


@pytest.mark.parametrize("new", [1, 60])
def test_attend_scales_that_are_not_powers_of_two(dq, new):
    b = Batch(dq, [200, 90], 2, 64, 32, seed=7)
    b.fill()
    for i, t in ((0, b.cache.k_scale), (1, b.cache.v_scale)):
        b.scales[i] = (b.scales[i] * b.rng.uniform(1, 2, b.scales[i].shape)).astype(np.float32)
        t.copy_(dev(b.scales[i]))
    check_attend(dq, b, [new, new], 8, "bf16")


@pytest.mark.parametrize("new", [1, 60])
def test_attend_pages_of_zeros_keep_their_weight(dq, new):
    """Values appended as zeros stand at the least scale; their keys count all the same."""
    b = Batch(dq, [210, 70], 2, 128, 16, seed=14)
    b.fill()
    for at in b.table[0, 2:9]:
        b.codes[1][at] = np.where(np.isnan(b.codes[1][at]), np.nan, 0.0)
        b.scales[1][at] = 2.0 ** -100
    b.cache.v.copy_(dev(b.codes[1].astype(np.float32)).to(torch.float8_e4m3fn))
    b.cache.v_scale.copy_(dev(b.scales[1]))
    check_attend(dq, b, [new, new], 4, "bf16")
    check_attend(dq, b, [new, new], 4, "bf16", window=100)


@pytest.mark.parametrize("hint", [1, MANY])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_stays_in_its_workspace(dq, dim, hint):
    from quantized_weight_dequantization_gb300 import _attention
    b = Batch(dq, [2000, 300, 1, 700], 4, dim, 32, seed=17)
    b.fill()
    new = [150, 40, 1, 0]
    q = dev(b.rng.standard_normal((191, 12, dim)).astype(np.float32), torch.bfloat16)
    cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    args = (b.cache, q, dev(b.table), dev(np.array(b.lens, np.int32)), cu, hint)
    ws, after = guarded(_attention._attention_need(191, 4, 12, 4, dim))
    out = dq.kv8_attention(*args, workspace=ws)
    assert bool((after == 0xA5).all()) and not bool(ws[:2048].any())
    assert torch.equal(out, dq.kv8_attention(*args))


@pytest.mark.parametrize("new", [1, 40])
def test_attend_captured_graph_outlives_a_larger_call(dq, new):
    """A larger call grows the stream's workspace; a graph captured before keeps its own."""
    b = Batch(dq, [700, 90], 2, 128, 64, seed=15)
    b.fill()
    q = dev(b.rng.standard_normal((2 * new, 4, 128)).astype(np.float32), torch.bfloat16)
    table, lens = dev(b.table), dev(np.array(b.lens, np.int32))
    cu = dev(np.array([0, new, 2 * new], np.int32))
    hint = 1 if new == 1 else MANY
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = dq.kv8_attention(b.cache, q, table, lens, cu, hint)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = dq.kv8_attention(b.cache, q, table, lens, cu, hint)
        many = torch.zeros(100000, 4, 128, dtype=torch.bfloat16, device="cuda")
        far = dev(np.array([0, 99990, 100000], np.int32))
        dq.kv8_attention(b.cache, many, table, lens, far, MANY)
        torch.cuda.synchronize()
        spoil = [torch.full((20 << 20,), 0x7F, dtype=torch.uint8, device="cuda")
                 for _ in range(4)]  # what was given back would be taken by these
        graph.replay()
        torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((x == 0x7F).all()) for x in spoil)


@pytest.mark.parametrize("new", [1, 5, 70])
def test_attend_on_another_stream_repeats_bit_for_bit(dq, new):
    b = Batch(dq, [3000, 90, 1500], 2, 128, 64, seed=8)
    b.fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = b.rng.bit_generator.state
    runs = []
    for stream in (None, side, side, None):
        b.rng.bit_generator.state = state
        torch.cuda.synchronize()
        runs.append(check_attend(dq, b, [new] * 3, 8, "bf16", stream=stream))
    torch.cuda.synchronize()
    for r in runs[1:]:
        for x, y in zip(r, runs[0]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("new", [1, 60])
def test_attend_page_that_holds_no_number_reaches_only_rows_that_see_it(dq, new):
    b = Batch(dq, [96, 96], 2, 64, 16, seed=12)
    b.fill()
    b.cache.v_scale[int(b.table[0, 5]), 1] = float("nan")  # keys 80 .. 95 of sequence 0
    q = dev(b.rng.standard_normal((2 * new, 4, 64)).astype(np.float32), torch.bfloat16)
    cu = dev(np.array([0, new, 2 * new], np.int32))
    out = dq.kv8_attention(b.cache, q, dev(b.table), dev(np.array([96, 96], np.int32)), cu,
                           1 if new == 1 else MANY)
    seen = torch.arange(2 * new, device="cuda") < new
    seen &= torch.arange(2 * new, device="cuda") + 96 - new >= 80
    broken = out.isnan().any(-1)
    assert torch.equal(broken[:, 2:], seen[:, None].expand(-1, 2)) and not broken[:, :2].any()


@pytest.mark.parametrize("new", [1, 60])
def test_attend_pages_that_do_not_exist_are_not_seen_and_counted(dq, new):
    b = Batch(dq, [200], 1, 64, 16, seed=13)
    b.fill()
    lens = dev(np.array([200], np.int32))
    q = dev(b.rng.standard_normal((new, 2, 64)).astype(np.float32), torch.bfloat16)
    cu = dev(np.array([0, new], np.int32))
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    hint = 1 if new == 1 else MANY
    want, lse = dq.kv8_attention(b.cache, q, dev(b.table), lens, cu, hint, return_lse=True,
                                 bad=bad)
    assert int(bad.item()) == 0
    for hole in (-1, b.pages, 1 << 30):
        t = b.table.copy()
        t[0, 2] = hole
        got, lse2 = dq.kv8_attention(b.cache, q, dev(t), lens, cu, hint, return_lse=True, bad=bad)
        assert int(bad.item()) > 0
        bad.zero_()
        assert torch.isfinite(got.float()).all() and (lse2 < lse).all()
    # a table narrower than the sequence
    got, lse2 = dq.kv8_attention(b.cache, q, dev(b.table[:, :4]), lens, cu, hint, return_lse=True,
                                 bad=bad)
    assert int(bad.item()) > 0 and torch.isfinite(got.float()).all() and (lse2 < lse).all()


def test_cache_past_4_gib(dq):
    """Codes past byte 2^32 of the cache, written and read."""
    pages, kv, page, dim = 70000, 8, 64, 128
    cache = dq.KV8Cache.empty(pages, kv, page, dim)
    assert cache.k.numel() > 2 ** 32
    rng = np.random.default_rng(14)
    table = np.array([[pages - 1, 3, pages - 2], [pages - 3, pages - 4, 0]], np.int32)
    lens = np.array([150, 70], np.int32)
    cu = np.array([0, 150, 220], np.int32)
    x = [dev(rng.standard_normal((220, kv, dim)).astype(np.float32), torch.bfloat16)
         for _ in range(3)]
    dq.kv8_append(cache, x[0], x[1], dev(table), dev(lens), dev(cu))
    small = dq.KV8Cache.empty(6, kv, page, dim)
    near = np.array([[5, 3, 4], [2, 1, 0]], np.int32)
    dq.kv8_append(small, x[0], x[1], dev(near), dev(lens), dev(cu))
    for q, c, n in ((x[2], dev(cu), MANY), (x[2], dev(cu), 1), (x[2][[149, 219]], None, 1)):
        a = dq.kv8_attention(cache, q, dev(table), dev(lens), c, n)
        b = dq.kv8_attention(small, q, dev(near), dev(lens), c, n)
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_append_and_attend_together(dq):
    """Norm and rotation, append, attention over several steps, against the definition of the
    whole in 64 bits on what the cache holds."""
    rng = np.random.default_rng(15)
    b = Batch(dq, [90, 41, 64], 2, 128, 32, seed=16)
    cos, sin = tables(100, 128, rng)
    lens = [0, 0, 0]
    for new in ([70, 33, 60], [1, 1, 1], [1, 1, 1], [18, 6, 2]):
        lens = [n + m for n, m in zip(lens, new)]
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
        qkv = dev(rng.standard_normal((int(cu[-1]), 12, 128)).astype(np.float32), torch.bfloat16)
        w = dev((1 + 0.2 * rng.standard_normal(128)).astype(np.float32), torch.bfloat16)
        q, k = dq.qk_norm_rope(qkv[:, :8], qkv[:, 8:10], w, w, dev(cos), dev(sin), dev(pos))
        args = dev(b.table), dev(np.array(lens, np.int32)), dev(cu)
        dq.kv8_append(b.cache, k, qkv[:, 10:], *args)
        for i, x in enumerate((k, qkv[:, 10:])):
            oracle_attn.append(b.codes[i], b.scales[i], host(x), None, None, b.table, lens, cu,
                               False)
        b.check()
        out = dq.kv8_attention(b.cache, q, *args)
        want, _, size, reach = oracle_attn.attend(
            host(q), b.codes[0], b.codes[1], b.scales[0], b.scales[1], b.table, lens, cu,
            128 ** -0.5, True, 0)
        close(host(out), want, (2.0 ** -10 + 2.0 ** -17 * reach[..., None]) * size
              + U["bf16"] * np.abs(want), "together")


def test_binding_refusals(dq):
    c = dq.KV8Cache.empty(4, 2, 16, 64)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="page holds"):
        dq.KV8Cache.empty(4, 2, 48, 64)
    with pytest.raises(ValueError, match="head_dim"):
        dq.KV8Cache.empty(4, 2, 16, 96)
    with pytest.raises(TypeError, match="expected"):
        dq.KV8Cache(c.k.view(torch.int8), c.v, c.k_scale, c.v_scale)
    with pytest.raises(ValueError, match="k_scale"):
        dq.KV8Cache(c.k, c.v, c.k_scale[:2], c.v_scale)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        dq.kv8_append(c, x.float(), x.float(), table, lens)
    with pytest.raises(TypeError, match="v: expected"):
        dq.kv8_append(c, x, x.half(), table, lens)
    with pytest.raises(ValueError, match="expected .tokens"):
        dq.kv8_append(c, x[:, :1], x[:, :1], table, lens)
    with pytest.raises(ValueError, match="cu says"):
        dq.kv8_append(c, x[:2], x[:2], table, lens)
    with pytest.raises(ValueError, match="contiguous"):
        dq.kv8_append(c, x.transpose(1, 2).contiguous().transpose(1, 2), x, table, lens)
    with pytest.raises(ValueError, match="block_table"):
        dq.kv8_append(c, x, x, table.long(), lens)
    with pytest.raises(dq.Dq4Error, match="ERR_ROTARY"):
        t = torch.zeros((4, 6), device="cuda")
        dq.kv8_append(c, x, x, table, lens, cos=t, sin=t)
    with pytest.raises(dq.Dq4Error, match="ERR_ALIGN"):
        y = torch.zeros(3 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 2, 64)
        dq.kv8_append(c, y, y, table, lens)
    with pytest.raises(ValueError, match="the cache has"):
        dq.kv8_attention(c, torch.zeros((3, 3, 64), dtype=torch.bfloat16, device="cuda"), table,
                         lens)
    with pytest.raises(dq.Dq4Error, match="ERR_N"):
        dq.kv8_attention(c, x, table, lens, window=-1)
    with pytest.raises(ValueError, match="workspace"):
        dq.kv8_attention(c, x, table, lens,
                         workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="out: expected shape"):
        dq.kv8_attention(c, x, table, lens, out=x[:2])
    with pytest.raises(ValueError, match="weight and k_weight"):
        dq.qk_norm_rope(x, x, x[0, 0], None)
    with pytest.raises(ValueError, match="positions"):
        t = torch.zeros((4, 8), device="cuda")
        dq.qk_norm_rope(x, x, None, None, t, t)
    with pytest.raises(ValueError, match="does not go"):
        dq.qk_norm_rope(x, x[:2], None, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dq.qk_norm_rope(x.cpu(), None, None, None)
    torch.cuda.synchronize()


def test_example_layer(dq):
    """The example's layer, with 4-bit projections around these operators.  A value of the cache
    is off by half a step of e4m3 at most, 2^-4 of it and 2^-5.8 in the mean square; outputs add
    many of them, so that their difference stays below the largest of one."""
    from examples import attention_layer

    assert max(attention_layer.main(steps=2, prompts=(200, 3, 64))) < 2.0 ** -4
