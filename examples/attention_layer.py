"""One attention layer with 4-bit projections, served from the 8-bit paged cache.

    python examples/attention_layer.py [--steps 4]

A batch of prompts of different lengths and then single tokens go through

    linear (4-bit weights) -> qk_norm_rope -> kv8_append -> kv8_attention -> linear

and every step's output is compared with the same layer on dequantized weights and an
unquantized cache, in 32 bits.  Prints the relative difference of each step: what the 8-bit
cache and 16-bit activations cost, about 3 % on random data.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_dequantization_gb300 as dq  # noqa: E402

DEV = torch.device("cuda")
HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 2048, 16, 8, 128, 64
DTYPE = torch.bfloat16


class Linear4:
    """A weight in nested 4-bit codes (rows x cols), random, of unit gain."""

    def __init__(self, rows, cols, gen):
        n = rows * cols
        packed, blocks, groups = dq.sizes(n, 64, 256)
        self.rows, self.cols = rows, cols
        self.args = (
            torch.randint(0, 256, (packed,), generator=gen, device=DEV, dtype=torch.uint8),
            torch.randint(0, 256, (blocks,), generator=gen, device=DEV, dtype=torch.uint8),
            torch.full((groups,), 0.5 / math.sqrt(cols), device=DEV),
            torch.linspace(-1, 1, 256, device=DEV), torch.linspace(-1, 1, 16, device=DEV),
            2.0 / math.sqrt(cols))

    def __call__(self, x):
        return dq.linear(x, *self.args, self.rows)

    def dense(self):
        return dq.dq4_nested(*self.args, self.rows * self.cols, out_dtype=torch.float32).view(
            self.rows, self.cols)


def rotation(positions):
    inv = 10000.0 ** (-torch.arange(0, DIM, 2, device=DEV, dtype=torch.float64) / DIM)
    angle = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


class Layer:
    def __init__(self, seqs, tokens, gen):
        self.qkv = Linear4((HEADS + 2 * KV_HEADS) * DIM, HIDDEN, gen)
        self.out = Linear4(HIDDEN, HEADS * DIM, gen)
        self.q_weight = torch.ones(DIM, device=DEV, dtype=DTYPE)
        self.k_weight = torch.ones(DIM, device=DEV, dtype=DTYPE)
        self.cos, self.sin = rotation(tokens)
        pages = -(-tokens // PAGE)
        self.cache = dq.KV8Cache.empty(seqs * pages, KV_HEADS, PAGE, DIM)
        self.table = torch.randperm(seqs * pages, generator=gen, device=DEV).to(
            torch.int32).view(seqs, pages)

    def __call__(self, x, positions, seq_lens, cu=None, max_new=1):
        """x: the new tokens' rows; seq_lens: the sequences' lengths with them."""
        rows = self.qkv(x).view(len(x), -1, DIM)
        q, k = dq.qk_norm_rope(rows[:, :HEADS], rows[:, HEADS:HEADS + KV_HEADS], self.q_weight,
                               self.k_weight, self.cos, self.sin, positions)
        dq.kv8_append(self.cache, k, rows[:, HEADS + KV_HEADS:], self.table, seq_lens, cu)
        y = dq.kv8_attention(self.cache, q, self.table, seq_lens, cu, max_new)
        return self.out(y.view(len(x), -1))


class Plain:
    """The same layer on dense weights, a list of keys and values, and torch in 32 bits."""

    def __init__(self, layer, seqs):
        self.layer, self.held = layer, [None] * seqs
        self.qkv, self.out = layer.qkv.dense(), layer.out.dense()

    def __call__(self, x, positions, counts):
        n = self.layer
        rows = (x.float() @ self.qkv.T).view(len(x), -1, DIM)
        qk = rows[:, :HEADS + KV_HEADS]
        qk = qk * (qk.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        c, s = n.cos[positions][:, None], n.sin[positions][:, None]
        a, b = qk.chunk(2, -1)
        qk = torch.cat((a * c - b * s, b * c + a * s), -1)
        v, outs, at = rows[:, HEADS + KV_HEADS:], [], 0
        for i, count in enumerate(counts):
            part = slice(at, at + count)
            at += count
            new = torch.stack((qk[part, HEADS:], v[part]))
            self.held[i] = new if self.held[i] is None else torch.cat((self.held[i], new), 1)
            keys, values = self.held[i].repeat_interleave(HEADS // KV_HEADS, 2)
            scores = torch.einsum("ihd,jhd->hij", qk[part, :HEADS], keys) / math.sqrt(DIM)
            later = torch.ones_like(scores[0], dtype=torch.bool).triu(len(keys) - count + 1)
            p = scores.masked_fill(later, float("-inf")).softmax(-1)
            outs.append(torch.einsum("hij,jhd->ihd", p, values))
        return torch.cat(outs).reshape(len(x), -1) @ self.out.T


def main(steps=4, prompts=(700, 33, 1, 256)):
    """Returns the relative difference of each step's output."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    layer = Layer(len(prompts), max(prompts) + steps, gen)
    plain = Plain(layer, len(prompts))
    lens, found = [0] * len(prompts), []
    for step in range(1 + steps):
        counts = list(prompts) if step == 0 else [1] * len(prompts)
        lens = [n + c for n, c in zip(lens, counts)]
        cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32,
                          device=DEV)
        positions = torch.cat([torch.arange(n - c, n, device=DEV) for n, c in zip(lens, counts)])
        x = torch.randn(sum(counts), HIDDEN, generator=gen, device=DEV).to(DTYPE)
        seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        if step == 0:
            y = layer(x, positions, seq_lens, cu, max(counts))
        else:
            y = layer(x, positions, seq_lens)
        want = plain(x, positions, counts)
        found.append(float((y.float() - want).norm() / want.norm()))
        print(f"step {step}: {sum(counts)} tokens, relative difference {found[-1]:.4f}")
    return found


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=4, help="single tokens after the prompts")
    main(ap.parse_args().steps)
