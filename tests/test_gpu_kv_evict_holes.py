"""q4_kv_evict on sequences some of whose pages do not exist: their tokens are
not there, so they neither stay nor count, and what is read and attended over
afterwards is the rows of the kept ones."""

import numpy as np
import pytest
import torch

from bit_group_wise_amd import kv, q4
from _kv import DEV, FMTS, UNIT, Pool

pytestmark = pytest.mark.gpu
BAD = [-1, 2 ** 31 - 1, -2 ** 31]


def keep_of(mass, there, budget, recent):
    """Kept positions of one sequence and head: of the tokens that are there, the last and the heaviest."""
    at = np.flatnonzero(there)
    if len(at) <= budget:
        return at.tolist()
    old = at[:len(at) - recent]
    key = sorted(old.tolist(), key=lambda t: (mass[t] != mass[t], -(mass[t] if mass[t] == mass[t] else 0), t))
    return sorted(key[:budget - recent]) + at[len(at) - recent:].tolist()


def run(fmt, dim, g, page, lens, holes, budget, recent, seed, heads=2, masses=None):
    """holes: pairs of sequence and place in its table."""
    rng = np.random.default_rng(seed)
    per = -(-budget // page)
    pool = Pool(fmt, g, dim, heads, page, lens, seed=seed, spare=len(lens) * per + 1)
    used = set(pool.table.reshape(-1).tolist())
    free = [p for p in rng.permutation(pool.cache.pages).tolist() if p not in used]
    there = [np.ones(n, dtype=bool) for n in lens]
    for i, (b, p) in enumerate(holes):
        pool.table[b, p] = (BAD + [pool.cache.pages])[i % 4]
        there[b][p * page:(p + 1) * page] = False
    new_table = np.array(free[:len(lens) * per]).reshape(len(lens), per)
    width = max(lens) + 3
    mass = (rng.random((len(lens), heads, width)) if masses is None else masses(rng, (len(lens), heads, width))).astype(np.float32)
    batch = kv.Batch(pool.dev_table(), torch.tensor(lens, dtype=torch.int32, device=DEV), max_len=max(lens))
    dev_new = torch.from_numpy(new_table.astype(np.int32)).to(DEV)
    print("holes", fmt, dim, g, page, lens, holes, budget, recent, flush=True)
    nl, nm, kept = kv.evict(pool.cache, batch, torch.from_numpy(mass).to(DEV), dev_new, budget, recent, width=budget + 5)
    torch.cuda.synchronize()
    count = [min(int(t.sum()), budget) for t in there]
    assert nl.tolist() == count
    hk, hm = kept.cpu().numpy(), nm.cpu().numpy()
    want = [[keep_of(mass[b, h], there[b], budget, recent) for h in range(heads)] for b in range(len(lens))]
    for b, m in enumerate(count):
        for h in range(heads):
            assert hk[b, h, :m].tolist() == want[b][h] and (hk[b, h, m:] == -1).all(), (b, h)
            assert np.array_equal(hm[b, h, :m], mass[b, h][want[b][h]], equal_nan=True) and (hm[b, h, m:] == 0).all()
    # the kept rows, read back and attended over by one more token each
    starts = torch.tensor(np.concatenate([[0], np.cumsum(count)]), dtype=torch.int32, device=DEV)
    after = kv.Batch(dev_new, nl, starts, tokens=sum(count), max_new=max(1, max(count)))
    rows = [t.double().cpu().numpy() for t in kv.read(pool.cache, after, torch.bfloat16)]
    q = torch.from_numpy(rng.standard_normal((len(lens), heads, dim))).to(DEV).bfloat16()
    out = kv.attention(pool.cache, kv.Batch(dev_new, nl), q).double().cpu().numpy()
    assert np.isfinite(out).all()
    first = 0
    for b, m in enumerate(count):
        for h in range(heads):
            k, v = (pool.values(half, b)[want[b][h], h].reshape(m, dim) for half in range(2))
            for half, x in enumerate((k, v)):
                assert (np.abs(rows[half][first:first + m, h] - x) <= UNIT[q4.BF16] * np.abs(x)).all()
            if not m:
                assert (out[b, h] == 0).all()
                continue
            x = k @ q[b, h].double().cpu().numpy() * dim ** -0.5
            p = np.exp(x - x.max())
            p /= p.sum()
            # scores are off by 2^-24 of the sum of |q k| a term, weights and values round once to fp16 each,
            # the result once to bfloat16; what fp16's subnormals lose is below 2^-27 of the values
            rel = 2 * 2.0 ** -24 * (dim + 16) * np.abs(k).max() * np.abs(q[b, h].double().cpu().numpy()).sum() + 2.0 ** -9
            tol = rel * (p @ np.abs(v)) + UNIT[q4.BF16] * np.abs(p @ v) + m * 2.0 ** -27 * np.abs(v).max()
            assert (np.abs(out[b, h] - p @ v) <= tol).all(), (b, h)
        first += m


@pytest.mark.parametrize("fmt", FMTS)
def test_holes(fmt):
    """Missing pages among the old tokens, the recent ones, at the end, and all of them; enough tokens or fewer than the budget."""
    run(fmt, 64, 32, 16, [100, 100, 41, 37, 40, 16, 0, 90],
        [(0, 1), (0, 4), (1, 6), (2, 0), (2, 2), (3, 1), (5, 0), (7, 0), (7, 1), (7, 2), (7, 3), (7, 4), (7, 5)],
        40, 11, seed=fmt)


@pytest.mark.parametrize("lens,holes,budget,recent", [
    ([70], [(0, 4)], 70, 5), ([70], [(0, 4)], 63, 63), ([70], [(0, 0)], 54, 0), ([70], [(0, 0)], 53, 0), ([70], [(0, 2)], 1, 0),
    ([70], [(0, 2)], 1, 1), ([1025], [(0, 3), (0, 64)], 900, 30), ([1025], [(0, p) for p in range(0, 65, 2)], 900, 30),
    ([5000], [(0, p) for p in range(1, 300, 7)], 4000, 100), ([9000, 70], [(0, 0), (0, 500), (1, 1)], 2500, 17)])
def test_holes_sizes(lens, holes, budget, recent):
    run(q4.INT4_ASYM, 64, 32, 16, lens, holes, budget, recent, seed=budget)


def test_holes_many_keys_a_thread():
    run(q4.FP4, 64, 64, 128, [36000, 17000], [(0, p) for p in range(0, 282, 9)] + [(1, 132)], 9000, 33, seed=2, heads=1,
        masses=lambda rng, shape: rng.integers(0, 9000, shape))


@pytest.mark.parametrize("kind", ["ties", "nan"])
def test_holes_masses(kind):
    """Equal masses, and tokens that count least of all (NaN) beside tokens that are not there."""
    def masses(rng, shape):
        m = rng.integers(0, 3, shape).astype(np.float32)
        if kind == "nan":
            m[rng.random(shape) < 0.8] = np.nan
        return m

    run(q4.INT4_SYM, 64, 64, 16, [700, 1300, 90], [(0, 2), (0, 30), (1, 0), (1, 80), (2, 5)], 300, 20, seed=4, masses=masses)
