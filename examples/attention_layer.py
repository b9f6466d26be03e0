"""One decoder attention layer served in 4 bits: weights and key/value cache.

The projections are quantized weights (q4.gemm / q4.gemv read them packed), the
keys and values of every token go into a paged 4-bit cache, attention reads
them there, and a request that outgrows its budget keeps the tokens that drew
the most attention.  Ragged prompts first, then one token a step:

    python examples/attention_layer.py [--seqs 4] [--steps 96] [--budget 192]

prints, at the end of the prompt and of the steps, how far the layer's output
is from the same layer over 16-bit keys and values (same weights, same tokens
kept), and the time of a step.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_group_wise_amd import kv, q4  # noqa: E402

DEV = "cuda:0"


class Layer:
    """Quantized projections of a layer with grouped heads."""

    def __init__(self, heads, group, dim, fmt=q4.NF4, g=64, seed=0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        self.heads, self.group, self.dim = heads, group, dim
        self.width = heads * group * dim
        rows = (heads * group + 2 * heads) * dim
        w = lambda n, k: torch.randn((n, k), generator=gen, device=DEV).mul_(k ** -0.5).half()  # noqa: E731
        self.qkv = q4.quantize(w(rows, self.width), fmt, g)
        self.out = q4.quantize(w(self.width, self.width), fmt, g)

    def project(self, x):
        """q, k, v [tokens, heads, dim]: slices of one product's output."""
        y = q4.gemm(x, self.qkv).view(x.shape[0], -1, self.dim)
        n = self.heads * self.group
        return y[:, :n], y[:, n:n + self.heads], y[:, n + self.heads:]

    def finish(self, att):
        return q4.gemm(att.view(att.shape[0], -1), self.out)


class Pool:
    """Which pages are free, and each request's table, on the host."""

    def __init__(self, cache, seqs, width):
        self.cache, self.free = cache, list(range(cache.pages))
        self.pages = [[] for _ in range(seqs)]
        self.table = torch.zeros((seqs, width), dtype=torch.int32)
        self.dev = torch.zeros((seqs, width), dtype=torch.int32, device=DEV)

    def grow(self, lens):
        for b, n in enumerate(lens):
            while len(self.pages[b]) * self.cache.page < n:
                self.pages[b].append(self.free.pop())
                self.table[b, len(self.pages[b]) - 1] = self.pages[b][-1]
        self.dev.copy_(self.table)

    def replace(self, b, pages):
        self.free += self.pages[b]
        self.pages[b] = pages
        self.table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)


def plain_attention(q, keys, values, group):
    """The newest tokens' attention over one request's 16-bit keys and values, in binary32."""
    k, v = (t.float().repeat_interleave(group, 0) for t in (keys, values))     # [q_heads, len, dim]
    n, L = q.shape[0], k.shape[1]
    x = torch.matmul(q.float().transpose(0, 1), k.transpose(1, 2)) * q.shape[-1] ** -0.5
    hidden = torch.arange(L, device=DEV)[None, :] > torch.arange(L - n, L, device=DEV)[:, None]
    p = torch.softmax(x.masked_fill(hidden, float("-inf")), -1)
    return torch.matmul(p, v).transpose(0, 1)                                    # [n, q_heads, dim]


def run(seqs=4, steps=96, budget=192, recent=32, heads=4, group=4, dim=128, page=32, fmt=q4.INT4_ASYM, g=32, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1)
    layer = Layer(heads, group, dim, seed=seed)
    lens = [budget // 2 + 17 * b for b in range(seqs)]                            # ragged prompts
    width = -(-(max(budget, max(lens)) + page) // page)
    cache = kv.alloc_cache(fmt, g, 2 * seqs * width, page, heads, dim, DEV)
    pool = Pool(cache, seqs, width)
    dev_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    mass = torch.zeros((seqs, heads, width * page), device=DEV)
    kept = [None] * seqs      # the 16-bit copy that the comparison attends over: (keys, values) [heads, len, dim]
    diff = []

    def compare(q, att, counts):
        first, num, den = 0, 0.0, 0.0
        for b, m in enumerate(counts):
            want = plain_attention(q[first:first + m], *kept[b], group)
            d = att[first:first + m].float() - want
            num, den, first = num + float(d.square().sum()), den + float(want.square().sum()), first + m
        diff.append((num / den) ** 0.5)

    # prompts
    pool.grow(lens)
    starts = torch.tensor([sum(lens[:b]) for b in range(seqs + 1)], dtype=torch.int32, device=DEV)
    prompt = kv.Batch(pool.dev, dev_lens, starts, tokens=sum(lens), max_new=max(lens))
    x = torch.randn((sum(lens), layer.width), generator=gen, device=DEV).bfloat16()
    q, k, v = layer.project(x)
    kv.append(cache, prompt, k, v)
    att = kv.attention(cache, prompt, q, mass=mass)
    first = 0
    for b, n in enumerate(lens):
        kept[b] = (k[first:first + n].transpose(0, 1), v[first:first + n].transpose(0, 1))
        first += n
    compare(q, att, lens)
    x = layer.finish(att)[(starts[1:] - 1).long()]

    # one token a step; requests that outgrow the budget are cut to it
    step = kv.Batch(pool.dev, dev_lens)
    evicted = 0
    torch.cuda.synchronize()
    spent = 0.0
    for s in range(steps):
        t0 = time.perf_counter()
        over = [b for b in range(seqs) if lens[b] >= budget + page - 1]
        if over:
            new_pages = [[pool.free.pop() for _ in range(-(-budget // page))] for _ in over]
            at = torch.tensor(over, device=DEV)
            part = kv.Batch(pool.dev[at], dev_lens[at])
            new_table = torch.tensor(new_pages, dtype=torch.int32, device=DEV)
            new_lens, new_mass, where = kv.evict(cache, part, mass[at], new_table, budget, recent, width=mass.shape[2])
            dev_lens[at], mass[at] = new_lens, new_mass
            for i, b in enumerate(over):
                pool.replace(b, new_pages[i])
                lens[b] = budget
                rows = where[i].long()[:, :, None].expand(-1, -1, dim)
                kept[b] = tuple(torch.gather(t, 1, rows) for t in kept[b])
                evicted += 1
        lens = [n + 1 for n in lens]
        pool.grow(lens)
        dev_lens += 1
        q, k, v = layer.project(x)
        kv.append(cache, step, k, v)
        att = kv.attention(cache, step, q, mass=mass)
        x = layer.finish(att)
        torch.cuda.synchronize()
        spent += time.perf_counter() - t0
        for b in range(seqs):
            kept[b] = tuple(torch.cat((old, new[b][:, None]), 1) for old, new in zip(kept[b], (k, v)))
    compare(q, att, [1] * seqs)
    return {"prompt_difference": diff[0], "step_difference": diff[1], "evictions": evicted, "lens": lens,
            "us_per_step": 1e6 * spent / max(steps, 1), "mass": mass, "device_lens": dev_lens}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--steps", type=int, default=96)
    ap.add_argument("--budget", type=int, default=192)
    a = ap.parse_args()
    r = run(seqs=a.seqs, steps=a.steps, budget=a.budget)
    print(f"output against 16-bit keys and values: prompt {r['prompt_difference']:.3f}, "
          f"after {a.steps} steps and {r['evictions']} evictions {r['step_difference']:.3f} (relative)")
    print(f"lengths {r['lens']}, {r['us_per_step']:.0f} us a step")


if __name__ == "__main__":
    main()
