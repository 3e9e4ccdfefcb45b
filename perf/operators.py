"""Timed cases of the attention-side operators: query/key norm with rotation, the 8-bit paged
key/value cache's append, and the attention that reads it.

Each case runs either in a plain form (elementary torch operations in 32 bits) or through the
framework's entry points, on the same inputs.  ``exact`` gives the same outputs from the
operators' definitions in 64 bits.

The cache.  ``k_cache`` and ``v_cache`` are float8_e4m3fn [pages, kv_heads, page, head_dim];
``k_scale`` and ``v_scale`` are float32 [pages, kv_heads].  A stored value is code * scale, one
scale for each page of tokens and head.  ``block_table[b, j]`` is the page that holds tokens
j * page .. of sequence b; ``seq_lens[b]`` its length with this call's tokens; tokens
``cu[b] .. cu[b + 1] - 1`` of the call are its last ones (``cu`` is None for one each).

  append   k is rotated by its position; s = max(the page's scale if it holds earlier tokens,
           the least power of two with max|x| <= 448 s over the page's new tokens, 2^-100);
           codes = e4m3(x / s); earlier codes of the page become e4m3(code * old / s).
  attend   out_i = sum_j p_ij v_j / sum_j p_ij with p_ij = exp(scale q_i . k_j) over the keys j
           with pos_i - window < j <= pos_i; no key: zeros (and a log-sum of -infinity).
  norm     y = R(pos) (w * x / sqrt(mean x^2 + eps)) for each head of q and of k, R the rotation
           of the first ``rotary`` values; backward: dx and dw of the same.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0
MIN_EXP = -100
EPS = 1e-6


# ----------------------------------------------------------------- the cases
def _norm(name, tokens, heads, kv_heads, dim, rotary, dtype, interleaved=False, backward=False):
    return {"name": name, "op": "norm_backward" if backward else "norm", "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rotary": rotary, "dtype": dtype,
            "interleaved": interleaved}


def _append(name, seqs, new_lo, new_hi, old_hi, kv_heads, dim, page, dtype, rotary,
            interleaved=False):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi,
            "old_hi": old_hi, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "rotary": rotary, "interleaved": interleaved}


def _attend(name, seqs, new_lo, new_hi, kv_lo, kv_hi, heads, kv_heads, dim, page, dtype,
            window=0, lse=False):
    return {"name": name, "op": "attend", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi,
            "kv_lo": kv_lo, "kv_hi": kv_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype, "window": window, "lse": lse}


def listed():
    return [
        # one decoding step of four sequences at hidden size 4096: latency is all
        _norm("norm, 4 tokens", 4, 32, 8, 128, 128, "bf16"),
        # a prompt batch whose q and k are views of the fused projection's output
        _norm("norm, prompt", 8191, 32, 8, 128, 128, "bf16"),
        # fine-tuning on short rows: small heads, half of each rotated, neighbours paired
        _norm("norm backward, small heads", 2047, 16, 16, 64, 32, "f16", True, True),
        # a fine-tuning step of 16384 tokens at hidden size 4096
        _norm("norm backward, 16k tokens", 16384, 32, 8, 128, 128, "bf16", False, True),
        # one decoding step of 64 sequences: every append lands inside a partly filled page
        _append("append, 64 x 1 token", 64, 1, 1, 4096, 8, 128, 64, "bf16", 128),
        # prompts of uneven lengths after earlier turns, small pages
        _append("append, prompts", 7, 300, 4001, 1000, 8, 128, 16, "f16", 64, True),
        # one user's short conversation: the smallest decoding call
        _attend("attend, 1 x 777", 1, 1, 1, 777, 777, 32, 8, 128, 64, "bf16", 0, True),
        # a serving batch of uneven lengths
        _attend("attend, 64 x up to 8192", 64, 1, 1, 100, 8192, 32, 8, 128, 64, "bf16"),
        # two very long documents: the key axis has to be split
        _attend("attend, 2 x 131071", 2, 1, 1, 90001, 131071, 64, 8, 128, 128, "f16"),
        # checking five proposed tokens for each of 24 sequences under a sliding window
        _attend("attend, 24 x 5 windowed", 24, 5, 5, 3, 6000, 16, 4, 64, 16, "bf16", 1024),
        # a fresh prompt
        _attend("attend, prompt of 8192", 1, 8192, 8192, 8192, 8192, 32, 8, 128, 64, "bf16"),
        # uneven chunks of prompts over what the cache holds already, small heads
        _attend("attend, chunks over 16k", 5, 1, 1025, 700, 16411, 16, 8, 64, 32, "f16", 0,
                True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    rotary = rng.choice([dim, dim // 2, dim // 2 + 8])
    interleaved = rng.random() < 0.4
    if op in ("norm", "norm_backward"):
        tokens = _log(rng, 1, min(16384, 16384 * 40 * 128 // ((heads + kv_heads) * dim)))
        return {k: v for k, v in _norm("", tokens, heads, kv_heads, dim, rotary, dtype,
                                       interleaved, op == "norm_backward").items() if k != "name"}
    seqs = _log(rng, 1, 96)
    if op == "append":
        new_hi = _log(rng, 1, max(2, 12000 // seqs))
        c = _append("", seqs, rng.choice([1, new_hi]), new_hi, _log(rng, 1, 5000), kv_heads, dim,
                    page, dtype, rotary, interleaved)
    else:
        kind = rng.choice(["decode", "few", "prompt"])
        window = rng.choice([0, 0, 1, 257, 4096])
        if kind == "decode":
            new_hi, kv_hi = 1, _log(rng, 5, max(6, min(131072, 500000 * 8 // (seqs * kv_heads))))
        elif kind == "few":
            new_hi, kv_hi = _log(rng, 2, 24), _log(rng, 5, max(6, min(30000, 160000 // seqs)))
        else:
            seqs = _log(rng, 1, 8)
            most = 32 * 8192 * 8192 / (heads * seqs)
            new_hi = _log(rng, 25, max(26, min(8192, int(math.sqrt(most)))))
            kv_hi = _log(rng, new_hi, max(new_hi + 1, min(20000, int(most / new_hi))))
        c = _attend("", seqs, rng.choice([1, new_hi]), new_hi, rng.choice([1, kv_hi]), kv_hi,
                    heads, kv_heads, dim, page, dtype, window, rng.random() < 0.5)
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(case):
    """The new tokens and the lengths with them, one of each for a sequence; the first sequence
    has the largest, the others lie evenly between the bounds."""
    rng = random.Random(case["seqs"])
    new = [case["new_hi"]] + [rng.randint(case["new_lo"], case["new_hi"])
                              for _ in range(case["seqs"] - 1)]
    if case["op"] == "append":
        old = [case["old_hi"]] + [rng.randint(0, case["old_hi"]) for _ in range(case["seqs"] - 1)]
        return new, [n + o for n, o in zip(new, old)]
    full = [case["kv_hi"]] + [rng.randint(case["kv_lo"], case["kv_hi"])
                              for _ in range(case["seqs"] - 1)]
    return new, [max(n, f) for n, f in zip(new, full)]


def _pairs(n, length, window):
    """(query, key) pairs in sight, and keys that some query sees, of one sequence."""
    first = length - n
    low = [max(0, p - window + 1) if window else 0 for p in (first, length - 1)]
    if not window or window >= length:
        return n * (first + 1) + n * (n - 1) // 2, length
    pairs = sum(min(p + 1, window) for p in range(first, length))
    return pairs, length - low[0]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] in ("norm", "norm_backward"):
        values = case["tokens"] * (case["heads"] + hk) * d
        tables = case["tokens"] * (4 * case["rotary"] + 8)
        if case["op"] == "norm":
            return {"bytes": 2 * values * size + tables + 2 * d * size, "flops": 7 * values}
        return {"bytes": 3 * values * size + tables + 2 * d * (size + 4), "flops": 16 * values}
    new, full = _lengths(case)
    if case["op"] == "append":
        tokens = sum(new)
        pages = sum((f - 1) // case["page"] - (f - n) // case["page"] + 1
                    for n, f in zip(new, full))
        values = 2 * tokens * hk * d
        return {"bytes": values * (size + 1) + 2 * pages * hk * 8 + 4 * pages
                + tokens * 4 * case["rotary"], "flops": 5 * values}
    pairs = keys = 0
    for n, f in zip(new, full):
        p, k = _pairs(n, f, case["window"])
        pairs += p
        keys += k
    rows = sum(new) * case["heads"]
    pages = sum(-(-f // case["page"]) for f in full)
    return {"bytes": 2 * keys * hk * d + 8 * pages * hk + 4 * pages + rows * (2 * d * size + (
        4 if case["lse"] else 0)), "flops": 4 * pairs * case["heads"] * d}


# ---------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _tables(positions, rotary, device):
    inv = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=device) / rotary)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def _activations(shape, dtype, gen):
    """Projections as they come: unit normal, with a few channels ten times as large."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = torch.rand(shape[-2:], generator=gen, device="cuda") < 0.02
    return torch.where(loud, 10 * x, x).to(dtype)


def prepare(case, seed):
    gen = _generator(seed)
    dev = torch.device("cuda")
    dtype = DTYPES[case["dtype"]]
    d, hk = case["dim"], case["kv_heads"]
    s = dict(case)
    if case["op"] in ("norm", "norm_backward"):
        t, hq = case["tokens"], case["heads"]
        # q and k are views of one row of the fused projection, with v behind them
        fused = _activations((t, hq + 2 * hk, d), dtype, gen)
        s["q"], s["k"] = fused[:, :hq], fused[:, hq:hq + hk]
        s["q_weight"] = (1 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(dtype)
        s["k_weight"] = (1 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(dtype)
        s["cos"], s["sin"] = _tables(max(t, 4096), case["rotary"], dev)
        s["positions"] = (torch.arange(t, device=dev) if case["tokens"] > 64 else
                          torch.randint(0, 4096, (t,), generator=gen, device=dev))
        if case["op"] == "norm_backward":
            s["dq_out"] = torch.randn((t, hq, d), generator=gen, device=dev).to(dtype)
            s["dk_out"] = torch.randn((t, hk, d), generator=gen, device=dev).to(dtype)
        return s
    new, full = _lengths(case)
    b, page = case["seqs"], case["page"]
    width = max(-(-f // page) for f in full)
    held = [-(-f // page) for f in full]
    pages = sum(held) + 3
    table = torch.full((b, width), 0, dtype=torch.int32)
    at = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed) % (1 << 62)))
    done = 0
    for i, n in enumerate(held):
        table[i, :n] = at[done:done + n]
        done += n
    s["block_table"] = table.to(dev)
    s["seq_lens"] = torch.tensor(full, dtype=torch.int32, device=dev)
    one = all(n == 1 for n in new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = None if one else torch.tensor(cu, dtype=torch.int32, device=dev)
    s["max_new"], s["tokens"], s["max_len"] = max(new), cu[-1], max(full)
    # earlier tokens in the cache, and a scale that fits them
    for name in ("k", "v"):
        loud = 1 + 9 * (torch.rand((1, hk, 1, d), generator=gen, device=dev) < 0.02)
        x = torch.randn((pages, hk, page, d), generator=gen, device=dev, dtype=torch.float16)
        codes = (x * loud.half()).mul_(8).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s[name + "_cache"] = codes
        s[name + "_scale"] = torch.exp2(torch.randint(-4, -2, (pages, hk), generator=gen,
                                                      device=dev).float())
    if case["op"] == "append":
        s["cos"], s["sin"] = _tables(max(full), case["rotary"], dev)
        s["k"] = _activations((cu[-1], hk, d), dtype, gen)
        s["v"] = _activations((cu[-1], hk, d), dtype, gen)
        s["touched"] = max((f - 1) // page - (f - n) // page + 1 for n, f in zip(new, full))
    else:
        # slots past a sequence's end were never written: whatever is there is no number
        tail = torch.arange(page, device=dev)
        for name in ("k", "v"):
            codes = s[name + "_cache"].view(torch.uint8)
            last = s["block_table"][torch.arange(b, device=dev),
                                    (s["seq_lens"].long() - 1) // page].long()
            used = (s["seq_lens"].long() - 1) % page + 1
            gone = tail[None, :] >= used[:, None]
            codes[last] = torch.where(gone[:, None, :, None], torch.full_like(codes[:1], 0x7F),
                                      codes[last])
        s["q"] = _activations((cu[-1], case["heads"], d), dtype, gen)
        s["softmax_scale"] = 1 / math.sqrt(d)
    if own:
        import quantized_weight_dequantization_gb300 as dq

        s["cache"] = dq.KV8Cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------- the two forms
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import quantized_weight_dequantization_gb300 as dq

    if s["op"] == "norm":
        return dq.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos"], s["sin"],
                               s["positions"], EPS, s["interleaved"])
    if s["op"] == "norm_backward":
        return dq.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"],
                                        s["k_weight"], s["cos"], s["sin"], s["positions"], EPS,
                                        s["interleaved"])
    if s["op"] == "append":
        dq.kv8_append(s["cache"], s["k"], s["v"], s["block_table"], s["seq_lens"], s["cu"],
                      s["cos"], s["sin"], s["interleaved"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return dq.kv8_attention(s["cache"], s["q"], s["block_table"], s["seq_lens"], s["cu"],
                            s["max_new"], s["softmax_scale"], window=s["window"],
                            return_lse=s["lse"])


def _run_plain(s):
    if s["op"] == "norm":
        return (_plain_norm(s["q"], s["q_weight"], s), _plain_norm(s["k"], s["k_weight"], s))
    if s["op"] == "norm_backward":
        dq_, dqw = _plain_norm_backward(s["dq_out"], s["q"], s["q_weight"], s)
        dk_, dkw = _plain_norm_backward(s["dk_out"], s["k"], s["k_weight"], s)
        return dq_, dk_, dqw, dkw
    if s["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _rotate(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] values of x turned by the angles: neighbours paired, or the
    first half with the second."""
    half = cos.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _plain_norm(x, weight, s):
    cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
    f = x.float()
    y = f * (f.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.float()
    return _rotate(y, cos, sin, s["interleaved"]).to(x.dtype)


def _plain_norm_backward(dy, x, weight, s):
    cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
    f = x.float()
    rstd = (f.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = f * rstd
    g = _rotate(dy.float(), cos, -sin, s["interleaved"])
    dw = (g * xh).sum((0, 1))
    gw = g * weight.float()
    dx = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _token_starts(s):
    if s["cu"] is not None:
        return s["cu"].long()
    return torch.arange(s["seqs"] + 1, device=s["seq_lens"].device)


def _plain_append(s):
    page, dev = s["page"], s["seq_lens"].device
    cu = _token_starts(s)
    full = s["seq_lens"].long()
    start = full - (cu[1:] - cu[:-1])
    # each sequence's pages that get tokens; where it has fewer than most, its first again
    j = torch.arange(s["touched"], device=dev)[None] + start[:, None] // page
    j = torch.where(j * page < full[:, None], j, start[:, None] // page)
    ids = torch.gather(s["block_table"].long(), 1, j)
    pos = j[..., None] * page + torch.arange(page, device=dev)  # [seqs, touched, page]
    is_new = (pos >= start[:, None, None]) & (pos < full[:, None, None])
    is_old = pos < start[:, None, None]
    token = (cu[:-1, None, None] + pos - start[:, None, None]).clamp(0, s["tokens"] - 1)
    at = pos.clamp(max=s["cos"].shape[0] - 1)
    is_new, is_old = is_new[..., None, None], is_old[..., None, None]
    for name in ("k", "v"):
        x = s[name][token].float()  # [seqs, touched, page, heads, dim]
        if name == "k":
            x = _rotate(x, s["cos"][at][..., None, :], s["sin"][at][..., None, :],
                        s["interleaved"])
        amax = torch.where(is_new, x.abs(), 0.0).amax((2, 4))  # [seqs, touched, heads]
        frac, power = torch.frexp(amax)
        power = torch.where(frac <= 0.875, power - 9, power - 8).clamp(min=MIN_EXP)
        power = torch.where(amax > 0, power, MIN_EXP)
        fit = ((power + 127) << 23).view(torch.float32)  # 2^power, exactly
        fit = torch.where(amax.isfinite(), fit, float("nan"))
        scales = s[name + "_scale"]
        before = torch.where(is_old.any(2)[..., 0], scales[ids], 0.0)
        scale = torch.maximum(before, fit)
        codes = s[name + "_cache"].view(torch.uint8)
        held = codes[ids].transpose(2, 3)  # [seqs, touched, page, heads, dim]
        ratio = (before / scale)[:, :, None, :, None]
        value = torch.where(is_new, x / scale[:, :, None, :, None],
                            held.view(torch.float8_e4m3fn).float() * ratio)
        value = value.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[ids] = torch.where(is_new | is_old, value, held).transpose(2, 3)
        scales[ids] = scale
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_attend(s):
    dev, page, hk = s["q"].device, s["page"], s["kv_heads"]
    b, n, length, d = s["seqs"], s["max_new"], s["max_len"], s["dim"]
    group = s["heads"] // hk
    cu, full = _token_starts(s), s["seq_lens"].long()
    count = cu[1:] - cu[:-1]
    ids = s["block_table"].long()
    key = torch.arange(ids.shape[1] * page, device=dev)
    held = (key < full[:, None])[:, None, :, None]

    def values(name):
        x = s[name + "_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
        x = x * s[name + "_scale"][ids][..., None, None]
        return torch.where(held, x.transpose(1, 2).reshape(b, hk, -1, d), 0.0)

    i = torch.arange(n, device=dev)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["tokens"] - 1)].float()
    q = q.reshape(b, n, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * n, d)
    scores = torch.matmul(q, values("k").transpose(2, 3)).mul_(s["softmax_scale"])
    scores = scores.view(b, hk, group, n, -1)
    pos = (full - count)[:, None] + i  # [seqs, n]
    seen = (key <= pos[..., None]) & (key < full[:, None, None])
    if s["window"]:
        seen &= key > pos[..., None] - s["window"]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, hk, group * n, -1), values("v")).view(b, hk, group, n, d)
    out = torch.where(total > 0, out / total, 0.0)
    token = torch.arange(s["tokens"], device=dev)
    of = torch.searchsorted(cu, token, right=True) - 1
    out = out.permute(0, 3, 1, 2, 4)[of, token - cu[of]].reshape(s["tokens"], -1, d)
    out = out.to(s["q"].dtype)
    if not s["lse"]:
        return out
    lse = (top + total.log()).permute(0, 3, 1, 2, 4)[of, token - cu[of]]
    return out, lse.reshape(s["tokens"], -1)


# ---------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        return _exact_norm(s)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s)


def _turn64(x, positions, cos, sin, interleaved, sign):
    """x as complex pairs, times exp(+-i angle)."""
    half = cos.shape[1]
    z = torch.complex(cos.double()[positions], sign * sin.double()[positions])
    while z.dim() < x.dim():
        z = z.unsqueeze(-2)
    y = x.clone()
    if interleaved:
        w = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z
        y[..., :2 * half] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * z
        y[..., :half], y[..., half:2 * half] = w.real, w.imag
    return y


def _exact_norm(s):
    outs, grads = [], []
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"].double()
        size = torch.sqrt((x * x).sum(-1, keepdim=True) / s["dim"] + EPS)
        if s["op"] == "norm":
            outs.append(_turn64(x / size * w, s["positions"], s["cos"], s["sin"],
                                s["interleaved"], 1.0))
            continue
        g = _turn64(s["d%s_out" % n].double(), s["positions"], s["cos"], s["sin"],
                    s["interleaved"], -1.0)
        grads.append((g * x / size).sum((0, 1)))
        inner = (g * w * x).sum(-1, keepdim=True)
        outs.append(g * w / size - x * inner / (s["dim"] * size ** 3))
    return tuple(outs + grads)


def _e4m3_64(x):
    """The nearest value with four significant bits, ties to even, steps of at least 2^-9."""
    _, power = torch.frexp(x.abs())
    step = ((power.long() - 4).clamp(min=-9) + 1023 << 52).view(torch.float64)  # exactly 2^..
    return torch.round(x / step) * step


def _exact_append(s):
    new, full = _lengths(s)
    page, table, at = s["page"], s["block_table"].cpu().tolist(), 0
    outs = {n: s[n].double() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    for b, (n, f) in enumerate(zip(new, full)):
        pos = torch.arange(f - n, f, device=s["k"].device)
        for name in ("k", "v"):
            x = s[name][at:at + n].double()
            if name == "k":
                x = _turn64(x, pos, s["cos"], s["sin"], s["interleaved"], 1.0)
            codes, scales = outs[name + "_cache"], outs[name + "_scale"]
            for j in range((f - n) // page, (f - 1) // page + 1):
                lo, hi = max(f - n, j * page), min(f, (j + 1) * page)
                part = x[lo - (f - n):hi - (f - n)].transpose(0, 1)  # [heads, tokens, dim]
                top = part.abs().amax((1, 2)).clamp(min=E4M3_MAX * 2.0 ** MIN_EXP)
                fit = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
                old = scales[table[b][j]] if lo > j * page else torch.zeros_like(fit)
                scale = torch.maximum(old, fit)
                kept = lo - j * page
                block = codes[table[b][j]]
                block[:, :kept] = _e4m3_64(block[:, :kept] * (old / scale)[:, None, None])
                block[:, kept:hi - j * page] = _e4m3_64(part / scale[:, None, None])
                scales[table[b][j]] = scale
        at += n
    return outs["k_cache"], outs["v_cache"], outs["k_scale"], outs["v_scale"]


def _exact_attend(s):
    new, full = _lengths(s)
    page, d, hk = s["page"], s["dim"], s["kv_heads"]
    group, at, outs, sums = s["heads"] // hk, 0, [], []
    for b, (n, f) in enumerate(zip(new, full)):
        ids = s["block_table"][b, :-(-f // page)].long()
        k, v = ((s[x + "_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                 * s[x + "_scale"].double()[ids][..., None, None]).transpose(0, 1)
                .reshape(hk, -1, d)[:, :f] for x in ("k", "v"))
        step = max(1, (1 << 26) // (f * s["heads"]))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            q = s["q"][at + lo:at + hi].double().reshape(hi - lo, hk, group, d)
            first = max(0, f - n + lo - s["window"] + 1) if s["window"] else 0
            score = torch.einsum("ihgd,hjd->hgij", q, k[:, first:]) * s["softmax_scale"]
            j = torch.arange(first, f, device=q.device)
            i = torch.arange(f - n + lo, f - n + hi, device=q.device)[:, None]
            hide = (j > i) | (j <= i - s["window"] if s["window"] else j < 0)
            score = score.masked_fill(hide, float("-inf"))
            log = torch.logsumexp(score, -1)
            o = torch.einsum("hgij,hjd->ihgd", torch.exp(score - log[..., None]), v[:, first:])
            outs.append(o.reshape(hi - lo, -1, d))
            sums.append(log.permute(2, 0, 1).reshape(hi - lo, -1))
        at += n
    out = torch.cat(outs)
    return (out, torch.cat(sums)) if s["lse"] else out
