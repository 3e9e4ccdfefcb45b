"""Timed cases of the operators with 8-bit weights: the row quantizer with outlier columns, the
8-bit matrix product, the gradient of its input, and a mixture-of-experts layer.

Each case runs either in a plain form (elementary torch operations in 32 bits) or through the
framework's entry points, on the same inputs.  ``exact`` gives the same outputs from the
operators' definitions in 64 bits.

A weight is int8 codes ``CB`` [N, K] with a float32 scale for each row, ``SCB``: the value is
CB * SCB / 127.

  quantize  s = max |x| over a row's values below the threshold (0 if that is below 2^-100, NaN
            if one of them is no number); code = the integer nearest to RN32(x * RN32(127 / s)),
            within +-127.  A column with a value at or above the threshold is an outlier; the
            first ``max_outliers`` keep their values in 16 bits and have codes of 0.
  linear    y = s S / 127^2 sum_k code * CB + S / 127 sum_l outlier_l * CB[:, cols_l] + bias
  backward  dX = dY W, W the weight's values rounded to dY's type
  moe       the top_k experts e of each token by its logits (ties: the lowest), weights p their
            softmax (over the chosen ones if renormalized, else over all):
            y = sum_e p_e W2_e (silu(Wg_e x) * (Wu_e x)), Wg the first half of w1's rows
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = 2.0 ** -100
THRESHOLD = 6.0


# ----------------------------------------------------------------- the cases
def _quantize(name, rows, cols, dtype, outliers=0, most=64):
    """outliers: how many columns are loud; 0: no threshold."""
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype,
            "outliers": outliers, "most": most}


def _linear(name, rows, n, k, dtype, outliers=0, bias=False, most=64):
    return {"name": name, "op": "linear", "rows": rows, "n": n, "k": k, "dtype": dtype,
            "outliers": outliers, "bias": bias, "most": most}


def _backward(name, rows, n, k, dtype):
    return {"name": name, "op": "backward", "rows": rows, "n": n, "k": k, "dtype": dtype}


def _moe(name, tokens, hidden, inner, experts, top_k, dtype, renormalize=True):
    return {"name": name, "op": "moe", "tokens": tokens, "hidden": hidden, "inner": inner,
            "experts": experts, "top_k": top_k, "dtype": dtype, "renormalize": renormalize}


def listed():
    return [
        # one decoding step of one sequence: latency is all
        _quantize("quantize, 1 x 4096", 1, 4096, "bf16"),
        # a prompt batch before a projection, a few loud columns
        _quantize("quantize, 2048 x 14336, outliers", 2048, 14336, "f16", 21),
        # one token through a square projection
        _linear("linear, 1 x 4096 to 4096", 1, 4096, 4096, "f16"),
        # a decoding batch through an up projection, with its bias and outlier columns
        _linear("linear, 8 x 4096 to 11008", 8, 11008, 4096, "f16", 5, True),
        # tokens of an odd batch through a wide layer
        _linear("linear, 61 x 8192 to 28672", 61, 28672, 8192, "bf16"),
        # a short prompt
        _linear("linear, 512 x 4096 to 11008", 512, 11008, 4096, "bf16", 13),
        # prompts of a batch through the largest layer
        _linear("linear, 8191 x 4096 to 14336", 8191, 14336, 4096, "bf16", 0, True),
        # fine-tuning adapters over a frozen weight: a short batch, a long one
        _backward("backward, 256 x 4096 from 4096", 256, 4096, 4096, "bf16"),
        _backward("backward, 2047 x 4096 from 11008", 2047, 11008, 4096, "f16"),
        # one token through few large experts: every byte of two of them
        _moe("moe, 1 token, 2 of 8 experts", 1, 4096, 14336, 8, 2, "bf16"),
        # a decoding batch through many small experts
        _moe("moe, 16 tokens, 6 of 64 experts", 16, 2048, 1408, 64, 6, "bf16", False),
        # a decoding batch that needs all of the large experts
        _moe("moe, 23 tokens, 2 of 8 experts", 23, 4096, 14336, 8, 2, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear", "backward", "moe", "moe"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "quantize":
        cols = _log(rng, 64, 20000)
        if rng.random() < 0.7:
            cols = -(-cols // 16) * 16
        rows = _log(rng, 1, min(16384, 2048 * 14336 // cols))
        c = _quantize("", rows, cols, dtype, rng.choice([0, 0, 1, 7, 40]), rng.choice([16, 64]))
    elif op in ("linear", "backward"):
        k = 16 * _log(rng, 4, 1024)
        n = _log(rng, 64, min(28672, 8192 * 28672 // k))
        most = 8191 * 14336 * 4096 if op == "linear" else 2047 * 11008 * 4096
        rows = _log(rng, 1, max(2, min(8191, most // (n * k))))
        if op == "linear":
            c = _linear("", rows, n, k, rng.choice(["bf16", "f16", "f32"]),
                        rng.choice([0, 0, 1, 9, 30]), rng.random() < 0.5, rng.choice([32, 64]))
        else:
            c = _backward("", rows, -(-n // 8) * 8, k, dtype)
    else:
        tokens = _log(rng, 1, 32)
        experts = rng.choice([2, 5, 8, 16, 60, 64, 128])
        hidden = 16 * _log(rng, 16, 512)
        inner = 16 * _log(rng, 8, min(896, 8 * 4096 * 14336 // (16 * experts * hidden)))
        c = _moe("", tokens, hidden, inner, experts, rng.randint(1, min(8, experts)), dtype,
                 rng.random() < 0.5)
    return {key: v for key, v in c.items() if key != "name"}


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "quantize":
        m, k = case["rows"], case["cols"]
        kept = min(case["outliers"], case["most"])
        return {"bytes": m * k * (size + 1) + 4 * m + 2 * m * kept, "flops": 4 * m * k}
    if case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        kept = min(case["outliers"], case["most"])
        return {"bytes": m * k + n * k + m * n * size + 4 * (m + n) + 2 * m * kept
                + (n * size if case["bias"] else 0), "flops": 2 * m * n * (k + kept)}
    if case["op"] == "backward":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": m * n * size + n * k + m * k * size + 4 * n, "flops": 2 * m * n * k}
    t, h, i, e = case["tokens"], case["hidden"], case["inner"], case["experts"]
    # experts that some token chooses, on average
    used = e * (1 - (1 - case["top_k"] / e) ** t)
    return {"bytes": int(used * (3 * h * i + 4 * (2 * i + h))) + 2 * t * h * size + 4 * t * e
            + 8 * t * case["top_k"], "flops": 6 * t * case["top_k"] * h * i}


# ---------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _codes(shape, gen):
    """Codes of a weight's rows: normal, the largest of each near 127."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat, step = out.view(-1), 1 << 27
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.float16)
                   .mul_(32).round_().clamp_(-127, 127))
    return out


def _scales(shape, fan_in, gen):
    """Row scales for outputs near 1."""
    return (0.5 + torch.rand(shape, generator=gen, device="cuda")) * (4 / math.sqrt(fan_in))


def _activations(rows, cols, loud, dtype, gen):
    """Rows of a hidden state: normal, and ``loud`` columns with values past the threshold."""
    x = torch.randn((rows, cols), generator=gen, device="cuda") * 0.8
    if loud:
        which = torch.rand(cols, generator=gen, device="cuda").argsort()[:loud]
        x[:, which] *= 12
    return x.to(dtype)


def prepare(case, seed):
    gen = _generator(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        s["x"] = _activations(case["rows"], case["cols"], case["outliers"], dtype, gen)
    elif case["op"] == "linear":
        half = torch.float16 if dtype == torch.float32 else dtype
        x = _activations(case["rows"], case["k"], case["outliers"], half, gen)
        rows = _plain_quantize(x, THRESHOLD if case["outliers"] else 0.0, case["most"])
        s["codes"], s["scales"] = rows[:2]
        s["kept"], s["outliers_"] = rows[2:4] if case["outliers"] else (None, None)
        s["CB"] = _codes((case["n"], case["k"]), gen)
        s["SCB"] = _scales(case["n"], case["k"], gen)
        s["bias_"] = (torch.randn(case["n"], generator=gen, device="cuda").to(dtype)
                      if case["bias"] else None)
        if own:
            import quantized_weight_dequantization_gb300 as dq

            s["x"] = dq.Int8Rows(s["codes"], s["scales"], s["kept"], s["outliers_"], None)
    elif case["op"] == "backward":
        s["dy"] = (torch.randn((case["rows"], case["n"]), generator=gen, device="cuda")
                   * 1e-2).to(dtype)
        s["CB"] = _codes((case["n"], case["k"]), gen)
        s["SCB"] = _scales(case["n"], case["k"], gen)
    else:
        t, h, i, e = case["tokens"], case["hidden"], case["inner"], case["experts"]
        s["x"] = _activations(t, h, max(1, h // 500), dtype, gen)
        s["logits"] = torch.randn((t, e), generator=gen, device="cuda")
        s["w1"], s["s1"] = _codes((e, 2 * i, h), gen), _scales((e, 2 * i), h, gen)
        s["w2"], s["s2"] = _codes((e, h, i), gen), _scales((e, h), i, gen)
    return s


# ------------------------------------------------------------- the two forms
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import quantized_weight_dequantization_gb300 as dq

    if s["op"] == "quantize":
        rows = dq.int8_quantize(s["x"], THRESHOLD if s["outliers"] else 0.0, s["most"])
        return tuple(rows) if s["outliers"] else tuple(rows[:2])
    if s["op"] == "linear":
        return dq.int8_linear(s["x"], s["CB"], s["SCB"], s["bias_"], DTYPES[s["dtype"]])
    if s["op"] == "backward":
        return dq.int8_linear_backward(s["dy"], s["CB"], s["SCB"])
    return dq.int8_moe(s["x"], s["logits"], s["w1"], s["s1"], s["w2"], s["s2"], s["top_k"],
                       s["renormalize"], return_routing=True)


def _run_plain(s):
    if s["op"] == "quantize":
        return _plain_quantize(s["x"], THRESHOLD if s["outliers"] else 0.0, s["most"])
    if s["op"] == "linear":
        return _plain_linear(s)
    if s["op"] == "backward":
        w = (s["CB"].float() * s["SCB"][:, None] * _R127).to(s["dy"].dtype)
        return torch.matmul(s["dy"].float(), w.float()).to(s["dy"].dtype)
    return _plain_moe(s)


_R127 = 0.007874015718698502  # 1 / 127 in 32 bits


def _plain_quantize(x, threshold, most):
    f = x.float()
    size = f.abs()
    loud = size >= threshold if threshold else torch.zeros_like(f, dtype=torch.bool)
    top = torch.where(loud, 0.0, size).amax(1)
    scales = torch.where(top < TINY, 0.0, torch.where(top.isfinite(), top, float("nan")))
    inverse = torch.where(scales > 0, torch.full_like(scales, 127.0) / scales, 0.0)
    codes = torch.where(inverse[:, None] > 0, f * inverse[:, None], 0.0).round()
    codes = codes.clamp(-127, 127).to(torch.int8)
    if not threshold:
        return codes, scales
    flag = loud.any(0)
    count = flag.sum(dtype=torch.int32).view(1)
    k = x.shape[1]
    # outlier columns first, in their order; those past ``most`` are left as they are
    order = torch.where(flag, 0, k) + torch.arange(k, device=x.device)
    order = torch.cat((order.sort()[0], order.new_full((most,), 2 * k)))[:most]
    cols = torch.where(order < k, order, -1)
    kept = torch.zeros(k + 1, dtype=torch.bool, device=x.device)
    kept[cols] = True  # (-1: the entry behind the last column)
    codes = torch.where(kept[:k], torch.zeros_like(codes), codes)
    outliers = torch.where(cols >= 0, x[:, cols.clamp(min=0)], torch.zeros_like(x[:1, :1]))
    return codes, scales, cols, outliers, count


def _plain_linear(s):
    a, b = s["codes"], s["CB"]
    total = None
    for lo in range(0, s["k"], 1024):  # sums of 1024 products are exact in 32 bits
        part = torch.matmul(a[:, lo:lo + 1024].float(), b[:, lo:lo + 1024].float().t())
        total = part.to(torch.int32) if total is None else total.add_(part.to(torch.int32))
    y = total.float() * (s["scales"] / 127)[:, None] * (s["SCB"] / 127)
    if s["kept"] is not None:
        use = s["kept"] >= 0
        x = torch.where(use, s["outliers_"].float(), 0.0)
        y += torch.matmul(x, b[:, s["kept"].clamp(min=0)].float().t()) * (s["SCB"] / 127)
    if s["bias_"] is not None:
        y += s["bias_"].float()
    return y.to(DTYPES[s["dtype"]])


def _plain_route(s):
    logits, k = s["logits"], s["top_k"]
    ids = logits.sort(dim=1, descending=True, stable=True)[1][:, :k]
    p = (logits - logits.amax(1, keepdim=True)).exp()
    chosen = p.gather(1, ids)
    total = chosen.sum(1, keepdim=True) if s["renormalize"] else p.sum(1, keepdim=True)
    return ids.to(torch.int32), chosen / total


def _plain_moe(s):
    ids, weights = _plain_route(s)
    x, i = s["x"].float(), s["inner"]
    y = torch.zeros_like(x)
    for e in range(s["experts"]):
        share = torch.where(ids == e, weights, 0.0).sum(1, keepdim=True)
        both = torch.matmul(x, s["w1"][e].float().t()) * (s["s1"][e] / 127)
        gate, up = both[:, :i], both[:, i:]
        hidden = gate / (1 + (-gate).exp()) * up
        out = torch.matmul(hidden, s["w2"][e].float().t()) * (s["s2"][e] / 127)
        y += torch.where(share > 0, share * out, 0.0)
    return y.to(s["x"].dtype), ids, weights


# ---------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(s)
    if case["op"] == "linear":
        return _exact_linear(s)
    if case["op"] == "backward":
        return _exact_backward(s)
    return _exact_moe(s)


def _to32(x):
    """Rounded to 32 bits, in 64."""
    return x.float().double()


def _exact_quantize(s):
    x = s["x"].double()
    limit = THRESHOLD if s["outliers"] else math.inf
    below = x.abs() < limit
    scale = (x.abs() * below).amax(1)
    scale = scale * (scale >= TINY)
    step = _to32(127.0 / scale)  # (of a row of zeros: infinite, and every code 0)
    codes = torch.nan_to_num(torch.round(_to32(x * step[:, None])), nan=0.0).clamp(-127, 127)
    if not s["outliers"]:
        return codes, scale
    found = (~below).any(0).nonzero()[:, 0]
    kept = found[:s["most"]]
    codes[:, kept] = 0
    cols = torch.cat((kept, kept.new_full((s["most"] - len(kept),), -1)))
    outliers = x.new_zeros((len(x), s["most"]))
    outliers[:, :len(kept)] = x[:, kept]
    return codes, scale, cols, outliers, torch.tensor([len(found)], device=x.device)


def _exact_linear(s):
    a = s["codes"].double() * s["scales"].double()[:, None] / 127
    if s["kept"] is not None:
        for at, c in enumerate(s["kept"].tolist()):
            if c >= 0:
                a[:, c] = s["outliers_"][:, at].double()
    y = torch.empty((len(a), s["n"]), dtype=torch.float64, device=a.device)
    for lo in range(0, s["n"], 2048):
        w = s["CB"][lo:lo + 2048].double() * s["SCB"][lo:lo + 2048].double()[:, None] / 127
        y[:, lo:lo + 2048] = a @ w.t()
    return y if s["bias_"] is None else y + s["bias_"].double()


def _exact_backward(s):
    dx = 0
    for lo in range(0, s["n"], 2048):
        w = _to32(_to32(s["CB"][lo:lo + 2048].double() * s["SCB"][lo:lo + 2048].double()[:, None])
                  * _R127)
        dx = dx + s["dy"][:, lo:lo + 2048].double() @ w.to(s["dy"].dtype).double()
    return dx


def _exact_moe(s):
    t, i, k = s["tokens"], s["inner"], s["top_k"]
    logits = s["logits"].double().cpu()
    ids, weights = [], []
    for row in logits.tolist():
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        part = [math.exp(row[e] - row[order[0]]) for e in order]
        total = sum(part) if s["renormalize"] else sum(math.exp(v - row[order[0]]) for v in row)
        ids.append(order)
        weights.append([p / total for p in part])
    x = s["x"].double()
    y = torch.zeros_like(x)
    for e in range(s["experts"]):
        rows = [(n, w) for n in range(t) for c, w in zip(ids[n], weights[n]) if c == e]
        if not rows:
            continue
        which = torch.tensor([n for n, _ in rows], device=x.device)
        share = torch.tensor([w for _, w in rows], dtype=torch.float64, device=x.device)
        part = x[which]
        gate, up = (part @ (s["w1"][e, lo:lo + i].double() * (s["s1"][e, lo:lo + i, None].double()
                                                              / 127)).t() for lo in (0, i))
        hidden = gate * torch.sigmoid(gate) * up
        out = hidden @ (s["w2"][e].double() * (s["s2"][e, :, None].double() / 127)).t()
        y.index_add_(0, which, out * share[:, None])
    return (y, torch.tensor(ids, device=x.device),
            torch.tensor(weights, dtype=torch.float64, device=x.device))
