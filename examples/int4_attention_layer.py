"""An attention layer that lives in 4 bits: INT4 projections and a paged 4-bit
key/value cache, served step by step.

    python examples/int4_attention_layer.py [--seqs 8] [--prompt 500] [--new 64]

A step takes the new tokens of some sequences (a prompt, a part of one, drafted
tokens or one token each) through

    q, k, v = x Wqkv^T            gemv_int4 (dequant_int4 and a product for
                                  more than 64 tokens)
    q, k    = rotate(norm(q, k))  kv4_append, which also writes k and v into
                                  the cache
    o       = attention(q)        kv4_attention over the cache
    y       = o Wo^T              gemv_int4

with four launches for single tokens (five where long caches are split).  All
weights and inputs here are random.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_dequantization_amd as lt  # noqa: E402


class Int4Linear:
    """y = x W^T with W [rows, cols] in INT4: packed codes, fp16 scales and
    int8 zero-points per group of a row."""

    def __init__(self, packed, scales, zp, rows, cols, group):
        self.packed, self.scales, self.zp = packed, scales, zp
        self.rows, self.cols, self.group = rows, cols, group

    @classmethod
    def random(cls, rows, cols, group, gen):
        dev, groups = gen.device, rows * cols // group
        packed = torch.randint(0, 256, (rows * cols // 2,), dtype=torch.uint8, device=dev, generator=gen)
        scales = torch.rand(groups, device=dev, generator=gen).add_(0.5).mul_(0.2 / cols ** 0.5).half()
        zp = torch.randint(6, 10, (groups,), device=dev, generator=gen).to(torch.int8)
        return cls(packed, scales, zp, rows, cols, group)

    def __call__(self, x):
        shape = (self.rows, self.cols)
        if x.shape[0] <= 64:
            return lt.gemv_int4(self.packed, self.scales, self.zp, shape, self.group, x)
        # many tokens: the expanded weights pay for themselves
        w = lt.dequant_int4(self.packed, self.scales, self.zp, shape, self.group)
        return x @ w.to(x.dtype).T


class Sequences:
    """Lengths and pages of the sequences that share a cache."""

    def __init__(self, cache, n_seqs, most_tokens):
        self.page_tokens, self.device = cache.page_tokens, cache.pages.device
        self.lens = [0] * n_seqs
        width = -(-most_tokens // cache.page_tokens)
        self.table = torch.full((n_seqs, width), -1, dtype=torch.int32)
        self.free = list(range(cache.pages.shape[0]))[::-1]

    def step(self, new):
        """The batch in which sequence i gets new[i] more tokens (0: it waits)."""
        starts = [0]
        for i, n in enumerate(new):
            have, want = (-(-t // self.page_tokens) for t in (self.lens[i], self.lens[i] + n))
            for p in range(have, want):
                self.table[i, p] = self.free.pop()
            self.lens[i] += n
            starts.append(starts[-1] + n)
        up = lambda t: torch.as_tensor(t, dtype=torch.int32).to(self.device)  # noqa: E731
        return lt.Kv4Batch(up(starts), up(self.lens), up(self.table), starts[-1], max(new), max(self.lens))


class AttentionLayer:
    def __init__(self, hidden, heads, kv_heads, head_dim, cache, most_tokens, group=128, rotary=None, seed=0,
                 dtype=torch.float16):
        gen = torch.Generator(cache.pages.device).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.cache = heads, kv_heads, head_dim, cache
        self.qkv = Int4Linear.random((heads + 2 * kv_heads) * head_dim, hidden, group, gen)
        self.out = Int4Linear.random(hidden, heads * head_dim, group, gen)
        self.q_norm = torch.rand(head_dim, device=gen.device, generator=gen).add_(0.5).to(dtype)
        self.k_norm = torch.rand(head_dim, device=gen.device, generator=gen).add_(0.5).to(dtype)
        rotary = rotary or head_dim
        turn = 10000.0 ** (-torch.arange(0, rotary, 2, device=gen.device, dtype=torch.float64) / rotary)
        angle = torch.arange(most_tokens, device=gen.device, dtype=torch.float64)[:, None] * turn
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def __call__(self, x, batch, window=0, sinks=0):
        """x [n_tokens, hidden] of the batch's new tokens -> [n_tokens, hidden]."""
        rows = self.qkv(x).view(x.shape[0], self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], 1)   # views: nothing is copied
        q = lt.kv4_append(self.cache, batch, k, v, q, q_norm=self.q_norm, k_norm=self.k_norm, cos=self.cos,
                          sin=self.sin)
        o = lt.kv4_attention(self.cache, batch, q, window=window, sinks=sinks)
        return self.out(o.view(x.shape[0], -1))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, v in (("seqs", 8), ("prompt", 500), ("new", 64), ("hidden", 4096), ("heads", 32), ("kv-heads", 8),
                    ("head-dim", 128), ("page", 64), ("group", 64), ("window", 0)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args()
    most = a.prompt + a.new
    cache = lt.Kv4Cache.empty(a.seqs * -(-most // a.page), a.page, a.kv_heads, a.head_dim, a.group)
    layer = AttentionLayer(a.hidden, a.heads, a.kv_heads, a.head_dim, cache, most)
    seqs = Sequences(cache, a.seqs, most)
    gen = torch.Generator("cuda").manual_seed(1)

    def rows(n):
        return torch.randn(n, a.hidden, device="cuda", generator=gen).half()

    y = layer(rows(a.seqs * a.prompt), seqs.step([a.prompt] * a.seqs), a.window)   # prompts, all at once
    x = y[a.prompt - 1::a.prompt].contiguous()      # the newest token of each
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    batches = [seqs.step([1] * a.seqs) for _ in range(a.new)]
    layer(x, batches[0], a.window)                  # the first use loads the kernels
    start.record()
    for batch in batches:
        y = layer(x, batch, a.window)
    end.record()
    torch.cuda.synchronize()
    wide = 2 * 2 * a.kv_heads * a.head_dim
    four = cache.pages.shape[1] * cache.pages.shape[2] / a.page
    print("%d sequences of %d tokens: %.1f us a step; cache %d bytes a token (%d in 16 bits); output finite: %s" %
          (a.seqs, most, start.elapsed_time(end) * 1e3 / a.new, four, wide, bool(y.isfinite().all())))


if __name__ == "__main__":
    main()
