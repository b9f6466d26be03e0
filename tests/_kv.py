"""Plain 64-bit model of the 4-bit key/value cache, in numpy on the host, and
the caches that the tests of bit_group_wise_amd.kv run on: random codes and
scales in the rows that a sequence holds, NaN and garbage everywhere else."""

import numpy as np
import torch

from bit_group_wise_amd import kv, q4

DEV = "cuda:0"
NF4_TABLE = np.array([-1.0, -0.696, -0.525, -0.395, -0.284, -0.185, -0.091, 0.0, 0.079, 0.161, 0.246,
                      0.338, 0.441, 0.562, 0.720, 1.0], dtype=np.float32)
FP4_TABLE = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]) / 6.0
FP4_TABLE = FP4_TABLE.astype(np.float32)
TORCH = {q4.F16: torch.float16, q4.BF16: torch.bfloat16}
FMTS = [q4.INT4_SYM, q4.INT4_ASYM, q4.NF4, q4.FP4]
UNIT = {q4.F16: 2.0 ** -11, q4.BF16: 2.0 ** -8}   # largest relative error of one rounding


def levels(fmt, codes, zero):
    """Levels of codes [..., groups, g] less the zero-points [..., groups, 1]."""
    if fmt == q4.NF4:
        return NF4_TABLE[codes].astype(np.float64)
    if fmt == q4.FP4:
        return FP4_TABLE[codes].astype(np.float64)
    return codes.astype(np.float64) - (8 if fmt == q4.INT4_SYM else zero.astype(np.float64))


def unpack(b):
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def row_values(fmt, g, codes, scales, zeros):
    """float64 values [..., dim] of rows codes [..., dim/2]."""
    c = unpack(codes)
    groups = c.shape[-1] // g
    c = c.reshape(*c.shape[:-1], groups, g)
    z = None if zeros is None else unpack(zeros)[..., :groups, None]
    return (levels(fmt, c, z) * scales.astype(np.float64)[..., None]).reshape(*c.shape[:-2], groups * g)


def quantize_rows(fmt, g, x):
    """Codes, scales, zeros of binary32 rows x [n, dim]: the coding rules one value at a time."""
    n, dim = x.shape
    f = np.float32
    xg = x.astype(f).reshape(n, dim // g, g)
    zeros = None
    with np.errstate(all="ignore"):
        if fmt == q4.INT4_SYM:
            s = np.minimum(np.abs(xg).max(-1) / f(7), f(65504)).astype(np.float16)
            q = np.rint(xg / s.astype(f)[..., None])
            c = np.where(s[..., None] > 0, np.clip(q, -8, 7), 0) + 8
        elif fmt == q4.INT4_ASYM:
            lo, hi = np.minimum(xg.min(-1), f(0)), np.maximum(xg.max(-1), f(0))
            s = np.minimum((hi - lo) / f(15), f(65504)).astype(np.float16)
            z = np.where(s > 0, np.clip(np.rint(-lo / s.astype(f)), 0, 15), 0)
            c = np.where(s[..., None] > 0, np.clip(np.rint(xg / s.astype(f)[..., None]) + z[..., None], 0, 15), 0)
            zb = z.astype(np.uint8)
            if zb.shape[1] % 2:
                zb = np.pad(zb, ((0, 0), (0, 1)))
            zeros = zb[:, 0::2] | zb[:, 1::2] << 4
        else:
            s = np.abs(xg).max(-1)
            q = np.where(s[..., None] > 0, xg / s[..., None], f(0))
            tab = (NF4_TABLE if fmt == q4.NF4 else FP4_TABLE).astype(np.float64)
            d = np.abs(q.astype(np.float64)[..., None] - tab)
            c = d.argmin(-1)                       # the first of equal distances
            if fmt == q4.FP4:                      # ties between magnitudes go to the smaller one
                m = np.abs(np.abs(q.astype(np.float64))[..., None] - tab[:8]).argmin(-1)
                c = np.where((q < 0) & (m > 0), m + 8, m)
    c = c.astype(np.uint8).reshape(n, dim)
    return c[:, 0::2] | c[:, 1::2] << 4, s, zeros


class Pool:
    """A cache with given lengths: host arrays of every row's contents and the device cache."""

    def __init__(self, fmt, g, dim, heads, page, lens, seed, spare=3, width=None, pages=None, first_page=0,
                 scale=(0.03, 0.3)):
        rng = np.random.default_rng(seed)
        self.fmt, self.g, self.dim, self.heads, self.page, self.lens = fmt, g, dim, heads, page, list(lens)
        per = [-(-n // page) for n in lens]
        width = max(1, max(per)) if width is None else width
        pages = sum(per) + spare if pages is None else pages
        order = first_page + rng.permutation(pages - first_page)[:sum(per)]
        # entries past a sequence's pages are never followed
        table = rng.choice(np.array([-1, pages, 2 ** 31 - 1, -2 ** 31]), (len(lens), width)).astype(np.int64)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        groups, zb = dim // g, (dim // g + 1) // 2
        self.cache = kv.alloc_cache(fmt, g, pages, page, heads, dim, DEV)
        self.rows = []
        for w in ("k", "v"):
            tc, ts, tz = (getattr(self.cache, w + p) for p in ("_codes", "_scales", "_zeros"))
            tc.random_(0, 256)
            ts.fill_(float("nan"))
            if tz is not None:
                tz.fill_(255)
            per_seq = []
            for b, n in enumerate(lens):
                codes = rng.integers(0, 256, (n, heads, dim // 2), dtype=np.uint8)
                scales = rng.uniform(*scale, (n, heads, groups)).astype(np.float16 if fmt in (1, 2) else np.float32)
                scales[rng.random(scales.shape) < 0.02] = 0
                zeros = rng.integers(0, 256, (n, heads, zb), dtype=np.uint8) if fmt == q4.INT4_ASYM else None
                if n:
                    t = np.arange(n)
                    pg, sl = torch.from_numpy(table[b][t // page]).to(DEV), torch.from_numpy(t % page).to(DEV)
                    for to, x in ((tc, codes), (ts, scales), (tz, zeros)):
                        if x is not None:
                            to[pg, :, sl] = torch.from_numpy(x).to(DEV)
                per_seq.append((codes, scales, zeros, row_values(fmt, g, codes, scales, zeros)))
            self.rows.append(per_seq)

    def values(self, half, b):
        """float64 [len, heads, dim] of sequence b."""
        return self.rows[half][b][3]

    def dev_table(self):
        return torch.from_numpy(self.table.astype(np.int32)).to(DEV)

    def batch(self, new=None, max_len=None, max_new=None):
        lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        if new is None:
            return kv.Batch(self.dev_table(), lens, max_len=max_len)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        return kv.Batch(self.dev_table(), lens, starts, tokens=int(sum(new)),
                        max_new=max(new) if max_new is None else max_new, max_len=max_len)


def attention_ref(pool, new, q, scale, window=0, hidden=None):
    """out, the sum of P |V|, lse, mass [seqs][heads, len], and the largest
    scale * sum |q K| of the call; q float64 [tokens, q_heads, dim].
    hidden[b]: truth values of cached tokens that take no part."""
    T, hq, dim = q.shape
    G = hq // pool.heads
    out, mag, lse = np.zeros((T, hq, dim)), np.zeros((T, hq, dim)), np.full((T, hq), -np.inf)
    mass = [np.zeros((pool.heads, n)) for n in pool.lens]
    worst, first = 0.0, 0
    for b, (n, m) in enumerate(zip(pool.lens, new)):
        pos = np.arange(n - m, n)[:, None]
        t = np.arange(n)
        see = t <= pos
        if window:
            see &= t > pos - window
        if hidden is not None and hidden[b] is not None:
            see &= ~hidden[b]
        for h in range(pool.heads):
            K, V = pool.values(0, b)[:, h], pool.values(1, b)[:, h]
            for j in range(h * G, h * G + G):
                qq = q[first:first + m, j]
                x = np.where(see, qq @ K.T * scale, -np.inf)
                if n:
                    worst = max(worst, float((np.abs(qq) @ np.abs(K).T).max() * scale))
                top = x.max(-1, keepdims=True, initial=-np.inf)
                p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
                l = p.sum(-1, keepdims=True)
                p = np.where(l > 0, p / np.where(l > 0, l, 1), 0)
                with np.errstate(divide="ignore"):
                    lse[first:first + m, j] = np.where(l > 0, np.where(np.isfinite(top), top, 0.0) + np.log(l), -np.inf)[:, 0]
                out[first:first + m, j] = p @ V
                mag[first:first + m, j] = p @ np.abs(V)
                mass[b][h] += p.sum(0)
        first += m
    return out, mag, lse, mass, worst
