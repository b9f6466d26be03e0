"""q4_kv_attention where values differ much in size: what a row does not see
leaves it alone, and what it sees counts by its own size.

Every row is held to what that row sees.  Tolerances, from the arithmetic:
scores and softmax weights as in test_gpu_kv_attention (relative error 2 delta
+ 2^-18 of a weight, delta of the row's own scores); a weight and a value are
each rounded once to fp16 (2^-11 each), the result once to the output's type.
A row's largest product of weight and scale is held at 2^9 or more, values at
2^11 or more for the largest scale of their token, so what fp16's subnormals
lose (2^-25 each) is less than 2^-31 of the row's largest product of weight
and scale a token, at 16 levels 2^-27 times that; groups down to 2^-14 of
their token's largest lose nothing more."""

import numpy as np
import pytest
import torch

from bit_group_wise_amd import kv, q4
from _kv import DEV, FMTS, TORCH, UNIT, Pool, row_values

pytestmark = pytest.mark.gpu
TABLES = [q4.NF4, q4.FP4]
KINDS = ["prompt", "few"]


def set_scales(pool, half, b, scales):
    """Gives sequence b's keys (half 0) or values (1) these scales [len, heads, groups]."""
    codes, old, zeros, _ = pool.rows[half][b]
    scales = scales.astype(old.dtype)
    pool.rows[half][b] = (codes, scales, zeros, row_values(pool.fmt, pool.g, codes, scales, zeros))
    t = np.arange(pool.lens[b])
    pg, sl = torch.from_numpy(pool.table[b][t // pool.page]).to(DEV), torch.from_numpy(t % pool.page).to(DEV)
    (pool.cache.v_scales if half else pool.cache.k_scales)[pg, :, sl] = torch.from_numpy(scales).to(DEV)


def sized_pool(fmt, g, dim, heads, page, lens, seed, size):
    """A pool whose values have scales between half and all of size(n, rng) [n, 1 or heads, 1 or groups]."""
    pool = Pool(fmt, g, dim, heads, page, lens, seed=seed)
    rng = np.random.default_rng(seed + 1)
    for b, n in enumerate(lens):
        set_scales(pool, 1, b, rng.uniform(0.5, 1.0, (n, heads, dim // g)) * size(n, rng))
    return pool


def check(pool, new, act, q, window=0, roundings=2):
    """roundings: to fp16 that a weight times a value goes through."""
    qd = q.double().cpu().numpy()
    T, hq, dim = qd.shape
    G, scale = hq // pool.heads, dim ** -0.5
    print("fmt", pool.fmt, "g", pool.g, "dim", dim, "lens", pool.lens, "new", new, "heads", pool.heads, hq, "window",
          window, "act", act, flush=True)
    batch = pool.batch(None if all(m == 1 for m in new) else new)
    got = kv.attention(pool.cache, batch, q, window=window).double().cpu().numpy()
    assert np.isfinite(got).all()
    first, wants = 0, np.empty(qd.shape)
    for b, (n, m) in enumerate(zip(pool.lens, new)):
        t, pos = np.arange(n), np.arange(n - m, n)[:, None]
        see = (t <= pos) & ((t > pos - window) if window else True)
        s = pool.rows[1][b][1].astype(np.float64).max(-1)          # [len, heads]
        for j in range(hq):
            h = j // G
            K, V, qq = pool.values(0, b)[:, h], pool.values(1, b)[:, h], qd[first:first + m, j]
            x = np.where(see, qq @ K.T * float(np.float32(scale)), -np.inf)
            worst = np.where(see, np.abs(qq) @ np.abs(K).T, 0).max(-1) * scale
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref, mag, top = p @ V, p @ np.abs(V), (p * s[:, h]).max(-1)
            rel = 2 * (2.0 ** -24 * (dim + 16) * worst + 2.0 ** -20) + 2.0 ** -18 + roundings * 2.0 ** -11
            tol = rel[:, None] * mag + UNIT[act] * np.abs(ref) + n * 2.0 ** -27 * top[:, None]
            tol += 2.0 ** -25 if act == q4.F16 else 0.0
            wants[first:first + m, j] = ref
            over = np.abs(got[first:first + m, j] - ref) - tol
            assert (over <= 0).all(), f"sequence {b}, head {j}, row {np.unravel_index(over.argmax(), over.shape)}: " \
                                      f"{over.max()} past the tolerance"
        first += m
    return got, wants


def queries(tokens, heads, dim, act, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((tokens, heads, dim))).to(DEV).to(TORCH[act])


def small_and_big(fmt):
    return (2.0 ** -22, 2.0 ** 22) if fmt in TABLES else (2.0 ** -9, 2.0 ** 13)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 128)])
@pytest.mark.parametrize("fmt", FMTS)
def test_large_values_ahead(fmt, dim, g, kind):
    """Rows before the first large value see small ones only."""
    small, big = small_and_big(fmt)
    cases = {"prompt": (([150, 70], [150, 70], 37), ([200, 64], [70, 40], 170)),
             "few": (([75, 34], [3, 2], 74), ([75, 34], [4, 2], 33), ([200, 64], [60, 40], 180))}
    for lens, new, at in cases[kind]:
        pool = sized_pool(fmt, g, dim, 2, 16, lens, dim + g, lambda n, rng: np.where(np.arange(n) < at, small, big)[:, None, None])
        check(pool, new, q4.BF16, queries(sum(new), 2, dim, q4.BF16, 1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 5, 40])
@pytest.mark.parametrize("fmt", FMTS)
def test_large_values_past_the_window(fmt, window, kind):
    small, big = small_and_big(fmt)
    for new in {"prompt": ([60, 90],), "few": ([1, 1], [3, 2])}[kind]:
        pool = sized_pool(fmt, 64, 128, 2, 32, [170, 110], window,
                          lambda n, rng: np.where(np.arange(n) < n - 50, big, small)[:, None, None])
        check(pool, new, q4.BF16, queries(sum(new), 4, 128, q4.BF16, 2), window=window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
@pytest.mark.parametrize("dim,g", [(64, 32), (128, 32), (128, 64), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("fmt", FMTS)
def test_unequal_groups(fmt, dim, g, act, kind):
    """Groups of a row 2^14 apart, in an order that changes from token to token and head to head."""
    def size(n, rng):
        e = rng.integers(-14, 1, (n, 2, dim // g))
        e[..., 0], e[..., -1] = 0, -14
        return np.exp2(rng.permuted(e, axis=-1))

    new = {"prompt": [90, 41], "few": [1, 1]}[kind]
    pool = sized_pool(fmt, g, dim, 2, 16, [130, 41], 3, size)
    check(pool, new, act, queries(sum(new), 4, dim, act, 3))


NEW = [n for k in KINDS for n in {"prompt": ([90, 41],), "few": ([1, 1], [3, 2])}[k]]


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("fmt", TABLES)
def test_heavy_token_of_small_values(fmt, new):
    """Nearly all the weight on a token whose values are 2^44 times smaller than the others'."""
    small, big = small_and_big(fmt)
    at = 0
    pool = sized_pool(fmt, 32, 128, 2, 16, [130, 41], 5, lambda n, rng: np.where(np.arange(n) == at, small, big)[:, None, None])
    q = np.zeros((sum(new), 4, 128))
    first = 0
    for b, m in enumerate(new):
        for j in range(4):
            k = pool.values(0, b)[at, j // 2]
            q[first:first + m, j] = k * (100.0 * 128 ** 0.5 / (k @ k))
        first += m
    check(pool, new, q4.BF16, torch.from_numpy(q).to(DEV).to(torch.bfloat16))


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("size", [2.0 ** -58, 2.0 ** -30, 2.0 ** 30, 2.0 ** 55])
@pytest.mark.parametrize("fmt", TABLES)
def test_values_of_one_size(fmt, size, new):
    """Caches of values that are all tiny, or all large."""
    pool = sized_pool(fmt, 64, 128, 2, 32, [130, 41], 5, lambda n, rng: np.full((n, 1, 1), size))
    check(pool, new, q4.BF16, queries(sum(new), 4, 128, q4.BF16, 4))
