"""q4_kv_append, q4_kv_read and q4_kv_evict: bit for bit against the coding
rules, the dequantize rule and a plain selection on the host."""

import numpy as np
import pytest
import torch

import oracle
from bit_group_wise_amd import kv, q4
from _kv import DEV, FMTS, TORCH, Pool, quantize_rows, row_values

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def rows_of(cache, table, b, positions):
    """Host arrays [half][codes, scales, zeros] of these positions' rows, [n, heads, ...]."""
    t = np.asarray(positions)
    pg = torch.from_numpy(table[b][t // cache.page].astype(np.int64)).to(DEV)
    sl = torch.from_numpy(t % cache.page).to(DEV)
    got = []
    for w in ("k", "v"):
        parts = [getattr(cache, w + p) for p in ("_codes", "_scales", "_zeros")]
        got.append([None if p is None else p[pg, :, sl].cpu().numpy() for p in parts])
    return got


def fresh_cache(fmt, g, dim, heads, page, lens, seed, spare=2):
    """A cache of sentinel bytes and a table for these lengths."""
    rng = np.random.default_rng(seed)
    per = [max(1, -(-n // page)) for n in lens]
    pages = sum(per) + spare
    cache = kv.alloc_cache(fmt, g, pages, page, heads, dim, DEV)
    for w in ("k", "v"):
        for p in ("_codes", "_scales", "_zeros"):
            t = getattr(cache, w + p)
            if t is not None:
                t.view(torch.uint8).fill_(0xA5)
    order = rng.permutation(pages)[:sum(per)]
    table = np.full((len(lens), max(per)), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return cache, table


def snapshot(cache):
    return [getattr(cache, w + p).view(torch.uint8).clone() for w in ("k", "v") for p in ("_codes", "_scales", "_zeros")
            if getattr(cache, w + p) is not None]


def data(rng, n, heads, dim, act):
    """Rows of ordinary values, and among them rows of zeros, of one sign, tiny and outlying ones."""
    x = rng.standard_normal((n, heads, dim)).astype(np.float32)
    flat = x.reshape(n * heads, dim)
    kind = rng.integers(0, 12, n * heads)
    flat[kind == 0] = 0
    flat[kind == 1] = np.abs(flat[kind == 1])
    flat[kind == 2] = -np.abs(flat[kind == 2]) - 1
    flat[kind == 3] *= np.float32(2.0 ** -20)
    flat[kind == 4, 5] = 900.0
    flat[kind == 5] = np.rint(flat[kind == 5] * 2) / 2      # quotients on the ties between levels
    return torch.from_numpy(x).to(TORCH[act])


@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
@pytest.mark.parametrize("dim,g", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
def test_append(fmt, dim, g, act):
    """Prompts of several sequences, strided inputs: every stored bit, and nothing else touched."""
    rng = np.random.default_rng(dim + g + fmt)
    heads, page, lens, new = 3, 16, [40, 7, 33, 16], [37, 7, 1, 0]
    cache, table = fresh_cache(fmt, g, dim, heads, page, lens, seed=fmt)
    T = sum(new)
    k, v = data(rng, T, heads, dim, act), data(rng, T, heads, dim, act)
    fused = torch.zeros((T, 2 * heads + 1, dim + 8), dtype=TORCH[act], device=DEV)
    fused[:, :heads, :dim], fused[:, heads:2 * heads, :dim] = k.to(DEV), v.to(DEV)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    batch = kv.Batch(torch.from_numpy(table.astype(np.int32)).to(DEV),
                     torch.tensor(lens, dtype=torch.int32, device=DEV), starts, tokens=T, max_new=max(new))
    before = snapshot(cache)
    kv.append(cache, batch, fused[:, :heads, :dim], fused[:, heads:2 * heads, :dim])
    torch.cuda.synchronize()
    first = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for half, x in enumerate((k, v)):
            if not m:
                continue
            got = rows_of(cache, table, b, range(n - m, n))[half]
            xs = x[first:first + m].float().numpy().reshape(m * heads, dim)
            c, s, z = quantize_rows(fmt, g, xs)
            assert np.array_equal(got[0].reshape(c.shape), c), f"codes of sequence {b}"
            assert np.array_equal(got[1].reshape(s.shape), s), f"scales of sequence {b}"
            if z is not None:
                assert np.array_equal(got[2].reshape(z.shape), z), f"zeros of sequence {b}"
            if act == q4.F16:   # and the oracle's codes and scales
                oc, os_, _ = oracle.quantize(fmt, g, x[first:first + m].reshape(m * heads, dim).view(torch.int16).numpy().view(np.uint16))
                assert np.array_equal(c, oc) and np.array_equal(s.view(os_.dtype), os_)
        first += m
    # everything outside the new rows is as it was
    written = torch.zeros((cache.pages, page), dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, new)):
        for t in range(n - m, n):
            written[table[b][t // page], t % page] = True
    for a, b_ in zip(before, snapshot(cache)):
        same = (a == b_).cpu().all(-1).all(1)
        assert bool(same[~written].all())


@pytest.mark.parametrize("fmt,dim,g", [(q4.INT4_SYM, 128, 128), (q4.INT4_ASYM, 64, 32), (q4.NF4, 256, 64), (q4.FP4, 128, 32)])
def test_many_rows_are_as_few(fmt, dim, g):
    """One call of many tokens stores and reads the bits that calls of few do, pages that are missing included."""
    rng = np.random.default_rng(fmt)
    heads, page, lens = 8, 16, [1024 * 256 // dim + 5, 700 * 256 // dim + 9]
    many, table = fresh_cache(fmt, g, dim, heads, page, lens, seed=5)
    few, _ = fresh_cache(fmt, g, dim, heads, page, lens, seed=5)
    table[0, 3], table[1, 0] = -1, many.pages   # no such pages: nothing is stored, zeros are read
    tab = torch.from_numpy(table.astype(np.int32)).to(DEV)
    T = sum(lens)
    k, v = (torch.from_numpy(rng.standard_normal((T, heads, dim)).astype(np.float32)).to(torch.bfloat16).to(DEV) for _ in range(2))

    def batch(upto, new):
        starts = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device=DEV)
        return kv.Batch(tab, torch.tensor(upto, dtype=torch.int32, device=DEV), starts, tokens=sum(new), max_new=max(new))

    kv.append(many, batch(lens, lens), k, v)
    got = kv.read(many, batch(lens, lens), torch.bfloat16)
    at, ends = [0, 0], [0, lens[0]]
    while at != lens:
        new = [min(200, n - a) for n, a in zip(lens, at)]
        rows = torch.cat([torch.arange(e + a, e + a + n) for e, a, n in zip(ends, at, new)]).to(DEV)
        at = [a + n for a, n in zip(at, new)]
        kv.append(few, batch(at, new), k[rows], v[rows])
        for x, y in zip(got, kv.read(few, batch(at, new), torch.bfloat16)):
            assert torch.equal(x[rows].view(torch.int16), y.view(torch.int16))
    for a, b in zip(snapshot(many), snapshot(few)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_tokens_one_by_one(fmt):
    """A sequence grown token by token holds what one prompt of it holds."""
    rng = np.random.default_rng(fmt)
    n, heads, dim, g, page = 35, 2, 128, 128, 16
    k, v = (data(rng, n, heads, dim, q4.BF16).to(DEV) for _ in range(2))
    one, table = fresh_cache(fmt, g, dim, heads, page, [n], seed=3)
    two, _ = fresh_cache(fmt, g, dim, heads, page, [n], seed=3)
    tab = torch.from_numpy(table.astype(np.int32)).to(DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    kv.append(one, kv.Batch(tab, lens, torch.tensor([0, n], dtype=torch.int32, device=DEV), tokens=n, max_new=n), k, v)
    step = kv.Batch(tab, lens)
    for t in range(n):
        lens.fill_(t + 1)
        kv.append(two, step, k[t:t + 1], v[t:t + 1])
    for a, b in zip(snapshot(one), snapshot(two)):
        assert torch.equal(a, b)


def test_append_leaves_out():
    """Positions before the start, page numbers outside the pool and lengths past max_len write nothing there."""
    cache, table = fresh_cache(q4.INT4_ASYM, 32, 64, 2, 16, [40, 3], seed=1)
    tab = table.copy()
    tab[0, 1] = cache.pages          # positions 16..31 of sequence 0
    k = torch.randn((20 + 8, 2, 64), device=DEV).half()
    before = snapshot(cache)
    lens = torch.tensor([40, 3], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 20, 28], dtype=torch.int32, device=DEV)
    batch = kv.Batch(torch.from_numpy(tab.astype(np.int32)).to(DEV), lens, starts, tokens=28, max_new=20)
    kv.append(cache, batch, k, k)
    torch.cuda.synchronize()
    changed = (before[0] != snapshot(cache)[0]).any(-1).any(1).cpu()
    want = torch.zeros_like(changed)
    for t in range(32, 40):
        want[table[0][2], t % 16] = True
    for t in range(3):
        want[table[1][0], t] = True
    assert torch.equal(changed & ~want, torch.zeros_like(want))
    rk, rv = kv.read(cache, batch, torch.float16)
    assert bool((rk[:12] == 0).all()) and bool((rk[20:25] == 0).all()) and bool((rk[25:] != 0).any())


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 126, 2.0 ** -60, 2.0 ** -120, 2.0 ** -130])
@pytest.mark.parametrize("fmt", FMTS)
def test_append_bf16_range(fmt, scale):
    """bf16 rows far outside fp16's range: INT4 scales saturate or vanish, table formats keep them."""
    rng = np.random.default_rng(2)
    x = (torch.from_numpy(rng.standard_normal((9, 2, 64))).clamp(-1.9, 1.9) * scale).to(torch.bfloat16)
    cache, table = fresh_cache(fmt, 32, 64, 2, 16, [9], seed=1)
    batch = kv.Batch(torch.from_numpy(table.astype(np.int32)).to(DEV), torch.tensor([9], dtype=torch.int32, device=DEV),
                     torch.tensor([0, 9], dtype=torch.int32, device=DEV), tokens=9, max_new=9)
    kv.append(cache, batch, x.to(DEV), x.to(DEV))
    c, s, z = quantize_rows(fmt, 32, x.float().numpy().reshape(18, 64))
    for got in rows_of(cache, table, 0, range(9)):
        assert np.array_equal(got[0].reshape(c.shape), c) and np.array_equal(got[1].reshape(s.shape), s)
        assert z is None or np.array_equal(got[2].reshape(z.shape), z)


@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
@pytest.mark.parametrize("dim,g", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
def test_read(fmt, dim, g, act):
    pool = Pool(fmt, g, dim, 3, 32, [70, 1, 0, 32], seed=g + dim)
    new = [69, 1, 0, 32]
    k, v = kv.read(pool.cache, pool.batch(new), TORCH[act])
    first = 0
    for b, (n, m) in enumerate(zip(pool.lens, new)):
        for half, got in enumerate((k, v)):
            want = pool.values(half, b)[n - m:]
            # one binary32 product, one rounding
            want = torch.from_numpy(want.astype(np.float32)).to(TORCH[act])
            assert torch.equal(got[first:first + m].cpu(), want)
        first += m


# ------------------------------------------------------------------ eviction
def keep_of(mass, n, budget, recent):
    """Kept positions of one sequence and head."""
    if n <= budget:
        return list(range(n))
    key = [(-(m if m == m else -np.inf), m != m, t) for t, m in enumerate(mass[:n - recent].tolist())]
    return sorted(t for *_, t in sorted(key)[:budget - recent]) + list(range(n - recent, n))


def run_evict(fmt, dim, g, heads, page, lens, budget, recent, seed, masses=None, extra=7):
    rng = np.random.default_rng(seed)
    pool = Pool(fmt, g, dim, heads, page, lens, seed=seed, spare=len(lens) * -(-budget // page) + 1)
    used = set(pool.table[pool.table >= 0].tolist()) & set(range(pool.cache.pages))
    free = [p for p in rng.permutation(pool.cache.pages).tolist() if p not in used]
    per = -(-budget // page)
    new_table = np.array(free[:len(lens) * per]).reshape(len(lens), per)
    width = max(lens) + 3
    mass = rng.random((len(lens), heads, width)).astype(np.float32) if masses is None else masses(rng, (len(lens), heads, width))
    mass[..., max(lens):] = np.nan
    batch = kv.Batch(pool.dev_table(), torch.tensor(lens, dtype=torch.int32, device=DEV), max_len=max(lens))
    before = snapshot(pool.cache)
    print("evict", fmt, dim, g, heads, page, lens, budget, recent, flush=True)
    nl, nm, kept = kv.evict(pool.cache, batch, torch.from_numpy(mass).to(DEV),
                            torch.from_numpy(new_table.astype(np.int32)).to(DEV), budget, recent, width=budget + extra)
    torch.cuda.synchronize()
    assert nl.tolist() == [min(n, budget) for n in lens]
    kept, nm = kept.cpu().numpy(), nm.cpu().numpy()
    for b, n in enumerate(lens):
        m = min(n, budget)
        rows = rows_of(pool.cache, new_table, b, range(m)) if m else None
        for h in range(heads):
            want = keep_of(mass[b, h], n, budget, recent)
            assert kept[b, h, :m].tolist() == want and (kept[b, h, m:] == -1).all(), (b, h)
            assert np.array_equal(nm[b, h, :m], mass[b, h][want], equal_nan=True) and (nm[b, h, m:] == 0).all()
            for half in range(2):
                for part in range(3):
                    if rows is not None and rows[half][part] is not None:
                        assert np.array_equal(rows[half][part][:, h], pool.rows[half][b][part][want, h])
    # the old pages are as they were
    keep = torch.ones(pool.cache.pages, dtype=torch.bool)
    keep[new_table.reshape(-1)] = False
    for a, b_ in zip(before, snapshot(pool.cache)):
        assert torch.equal(a[keep], b_[keep])


@pytest.mark.parametrize("dim,g", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
def test_evict(fmt, dim, g):
    run_evict(fmt, dim, g, 3, 16, [100, 41, 40, 3, 0, 65], 40, 11, seed=dim + g)


@pytest.mark.parametrize("lens,budget,recent", [([2, 1], 1, 0), ([2], 1, 1), ([50], 49, 49), ([50], 49, 0), ([1025], 1024, 3),
                                                ([3000, 1500], 1, 0), ([5000], 4999, 100), ([2049, 2048, 2047], 1024, 1024),
                                                ([9000, 70], 2500, 17), ([33000], 16000, 1000)])
def test_evict_sizes(lens, budget, recent):
    run_evict(q4.INT4_ASYM, 64, 32, 2, 64, lens, budget, recent, seed=budget)


@pytest.mark.parametrize("fmt", [q4.INT4_ASYM, q4.NF4])
def test_evict_many_rows(fmt):
    run_evict(fmt, 256, 64, 8, 64, [5000, 4500], 4096, 64, seed=fmt)


def test_evict_many_keys_a_thread():
    run_evict(q4.FP4, 64, 64, 2, 128, [20000, 17000], 9000, 33, seed=2, masses=lambda rng, shape: rng.integers(0, 9000, shape).astype(np.float32))


def _ties(rng, shape):
    return rng.integers(0, 3, shape).astype(np.float32)


def _zeros(rng, shape):
    m = np.zeros(shape, dtype=np.float32)
    m[..., ::2] = -0.0
    return m


def _odd(rng, shape):
    m = rng.standard_normal(shape).astype(np.float32) * np.exp2(rng.integers(-140, 120, shape)).astype(np.float32)
    m[rng.random(shape) < 0.1] = np.inf
    m[rng.random(shape) < 0.1] = -np.inf
    m[rng.random(shape) < 0.2] = np.nan
    return m


def _close(rng, shape):
    """Numbers that differ in the last bits only."""
    return (np.float32(1.0).view(np.uint32) + rng.integers(0, 300, shape).astype(np.uint32)).view(np.float32)


@pytest.mark.parametrize("masses", [_ties, _zeros, _odd, _close])
def test_evict_masses(masses):
    run_evict(q4.INT4_SYM, 64, 64, 4, 16, [700, 1300, 90], 300, 20, seed=4, masses=masses)


def test_evict_refusals():
    pool = Pool(q4.INT4_SYM, 64, 64, 2, 16, [40], seed=1, spare=6)
    b = kv.Batch(pool.dev_table(), torch.tensor([40], dtype=torch.int32, device=DEV), max_len=40)
    mass = torch.zeros((1, 2, 48), device=DEV)
    new = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    for kw in (dict(budget=0, recent=0), dict(budget=8, recent=9), dict(budget=8, recent=-1), dict(budget=33, recent=0),
               dict(budget=8, recent=0, width=7)):
        with pytest.raises(q4.Q4Error):
            kv.evict(pool.cache, b, mass, new, **kw)
    with pytest.raises(q4.Q4Error):
        kv.evict(pool.cache, b, mass[..., :39].contiguous(), new, 8, 0)
    with pytest.raises(TypeError):
        kv.evict(pool.cache, b, mass.double(), new, 8, 0)
    with pytest.raises(TypeError):
        kv.append(pool.cache, pool.batch(), torch.zeros((1, 2, 64), device=DEV).half(), torch.zeros((1, 2, 64), device=DEV).bfloat16())
    with pytest.raises(ValueError):
        kv.append(pool.cache, pool.batch(), torch.zeros((2, 2, 64), device=DEV).half(), torch.zeros((2, 2, 64), device=DEV).half())
    with pytest.raises(q4.Q4Error):
        kv.alloc_cache(q4.NF4_DQ, 64, 4, 16, 2, 64, DEV)


def test_offsets_past_32_bits():
    """Rows more than 4 GiB into the pool: append, read back."""
    heads, dim, page = 8, 128, 64
    pages = 5 * 2 ** 30 // (heads * page * dim // 2)
    cache = kv.alloc_cache(q4.INT4_SYM, 64, pages, page, heads, dim, DEV)
    table = torch.tensor([[pages - 1, pages - 5]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([100], dtype=torch.int32, device=DEV)
    batch = kv.Batch(table, lens, torch.tensor([0, 100], dtype=torch.int32, device=DEV), tokens=100, max_new=100)
    x = torch.randn((100, heads, dim), device=DEV).half()
    kv.append(cache, batch, x, -x)
    k, v = kv.read(cache, batch, torch.float16)
    c, s, _ = quantize_rows(q4.INT4_SYM, 64, x.float().cpu().numpy().reshape(-1, dim))
    want = row_values(q4.INT4_SYM, 64, c, s, None).astype(np.float32)
    assert np.array_equal(k.float().cpu().numpy().reshape(-1, dim), torch.from_numpy(want).half().float().numpy())
    assert int((cache.k_codes[:pages - 5] != 0).sum()) == 0
