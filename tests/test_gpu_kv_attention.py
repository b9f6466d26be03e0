"""q4_kv_attention against a plain computation in 64 bits.

Tolerances, from the arithmetic.  Scores: products of exact 16-bit values and
levels summed in binary32 in any order, then a few more roundings, so a score
is off by at most delta = 2^-24 (dim + 16) * max sum |q K| * scale + 2^-20; a
softmax weight by 2 delta + 2^-18 relatively (numerator and denominator).
Output: weights and values may each be rounded once to fp16 (2^-11 each),
below fp16's normal range to multiples of 2^-24 of a weight scaled to at least
2^8 (2^-33 of the largest a token, at most 16 levels of the largest scale, 2^8
for scales between the largest and what it was scaled by: n 2^-21 max scale
bounds them), the result once to the output's type.  lse: delta + a rounding
of it.  Mass: a sum of weights, and binary32 additions to what was there."""

import numpy as np
import pytest
import torch

from bit_group_wise_amd import kv, q4
from _kv import DEV, FMTS, TORCH, UNIT, Pool, attention_ref

pytestmark = pytest.mark.gpu


def queries(rng, tokens, heads, dim, act, spread=1.0, pad=0):
    """fp16/bf16 queries on the device, rows further apart than they are long if pad, and as float64."""
    q = torch.from_numpy(rng.standard_normal((tokens, heads + pad, dim)) * spread).to(DEV).to(TORCH[act])
    q = q[:, :heads]
    return q, q.double().cpu().numpy()


def check(pool, new, act, q_heads, window=0, scale=None, spread=1.0, seed=0, pad=0, mass=True, batch=None,
          hidden=None, tag=""):
    rng = np.random.default_rng(seed + 77)
    tokens = int(sum(new))
    q, qd = queries(rng, tokens, q_heads, pool.dim, act, spread, pad)
    sc = pool.dim ** -0.5 if scale is None else scale
    if batch is None:
        batch = pool.batch(None if all(m == 1 for m in new) else new)
    width = max(pool.table.shape[1] * pool.page, 1) + 5
    m0 = rng.random((len(new), pool.heads, width)).astype(np.float32)
    md = torch.from_numpy(m0).to(DEV) if mass else None
    lse = torch.full((tokens, q_heads), 7.0, device=DEV)
    print(tag, "fmt", pool.fmt, "g", pool.g, "dim", pool.dim, "page", pool.page, "lens", pool.lens[:6], "new",
          list(new)[:6], "heads", pool.heads, q_heads, "window", window, flush=True)
    out = kv.attention(pool.cache, batch, q, scale=scale, window=window, mass=md, lse=lse)
    torch.cuda.synchronize()
    ref, mag, rl, rm, worst = attention_ref(pool, new, qd, float(np.float32(sc)), window, hidden)
    delta = 2.0 ** -24 * (pool.dim + 16) * worst + 2.0 ** -20
    rel = 2 * delta + 2.0 ** -18
    top = max([float(np.abs(r[1].astype(np.float64)).max()) for half in pool.rows for r in half if r[1].size] + [0.0])
    got = out.double().cpu().numpy()
    tol = (rel + 2 * 2.0 ** -11) * mag + UNIT[act] * np.abs(ref) + max(pool.lens) * 2.0 ** -21 * top + 2.0 ** -24
    assert np.isfinite(got).all(), "non-finite output"
    err = np.abs(got - ref) - tol
    assert (err <= 0).all(), f"out off at {np.unravel_index(err.argmax(), err.shape)}: {err.max()}"
    gl = lse.double().cpu().numpy()
    some = np.isfinite(rl)
    assert np.array_equal(some, np.isfinite(gl)) and (gl[~some] == -np.inf).all()
    assert (np.abs(gl[some] - rl[some]) <= delta + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl[some])).all(), "lse"
    if mass:
        gm = md.cpu().numpy().astype(np.float64)
        want = m0.astype(np.float64)
        for b, n in enumerate(pool.lens):
            want[b, :, :n] += rm[b]
            add = rm[b]
            tm = rel * add + 2.0 ** -22 * (want[b, :, :n] + add) + 2.0 ** -30
            assert (np.abs(gm[b, :, :n] - want[b, :, :n]) <= tm).all(), f"mass of sequence {b}"
            assert (gm[b, :, n:] == m0[b, :, n:]).all(), "mass past the length"
    return out, lse, md


@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
@pytest.mark.parametrize("dim,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("fmt", FMTS)
def test_token(fmt, dim, g, act):
    """One token a sequence: every format, width, group and type; ragged lengths, one token and none among them."""
    pool = Pool(fmt, g, dim, 2, 32, [75, 1, 0, 33, 310], seed=dim + g + fmt)
    check(pool, [1] * 5, act, 8, pad=1, seed=fmt)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 16, 17, 64])
def test_token_groups_and_pages(group, page):
    pool = Pool(q4.INT4_SYM, 64, 128, 3, page, [page, page + 1, page - 1, 2 * page + 15, 1], seed=group * page)
    check(pool, [1] * 5, q4.BF16, 3 * group, seed=group)


@pytest.mark.parametrize("dim,g,rows", [(64, 64, 64), (64, 32, 32), (64, 64, 33), (128, 128, 32), (128, 128, 17), (128, 32, 8),
                                        (128, 32, 5), (256, 128, 16), (256, 64, 8), (256, 32, 4), (256, 32, 3), (256, 32, 1)])
@pytest.mark.parametrize("fmt", [q4.INT4_ASYM, q4.NF4])
def test_token_rows(fmt, dim, g, rows):
    """As many rows as fill one, two or four column tiles, by one token's heads and by several tokens'."""
    pool = Pool(fmt, g, dim, 2, 32, [700, 45, 2], seed=rows)
    check(pool, [1, 1, 1], q4.F16, 2 * rows, seed=rows)
    check(pool, [rows, max(1, rows - 1), 1], q4.BF16, 2, seed=rows, window=100)


def test_many_sequences():
    """Sequences and heads enough to fill the card unsplit (of 6 and of 4 waves a workgroup), and beyond."""
    for seqs, heads in ((100, 4), (128, 4), (150, 4), (210, 4)):
        pool = Pool(q4.NF4, 64, 64, heads, 16, [530 + (7 * b) % 60 if b % 9 else b % 5 for b in range(seqs)], seed=seqs)
        check(pool, [1] * seqs, q4.BF16, 2 * heads, seed=seqs)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 1023, 1025, 5003])
@pytest.mark.parametrize("fmt", [q4.INT4_ASYM, q4.NF4])
def test_token_lengths(fmt, length):
    pool = Pool(fmt, 32, 64, 1, 16, [length, max(1, length // 2)], seed=length)
    check(pool, [1, 1], q4.F16, 4, seed=length)


@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
@pytest.mark.parametrize("dim,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("fmt", FMTS)
def test_prompt(fmt, dim, g, act):
    """Whole prompts and chunks of them: some rows before the cache's start (they see nothing)."""
    pool = Pool(fmt, g, dim, 2, 16, [70, 200, 3, 0, 129], seed=dim + g + fmt)
    check(pool, [70, 37, 5, 2, 65], act, 4, seed=fmt + 1)


@pytest.mark.parametrize("new", [2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 127, 130])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_chunk_sizes(group, new):
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 64, [new + 300, new, 2 * new + 1], seed=new)
    check(pool, [new, new, max(1, new - 1)], q4.BF16, 2 * group, seed=new)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 64, 100, 1000])
@pytest.mark.parametrize("fmt", [q4.INT4_ASYM, q4.FP4])
def test_window(fmt, window):
    pool = Pool(fmt, 32, 64, 2, 16, [400, 65, 7], seed=window)
    check(pool, [1, 1, 1], q4.F16, 8, window=window, seed=1)
    check(pool, [5, 3, 7], q4.F16, 8, window=window, seed=2)
    check(pool, [150, 65, 7], q4.BF16, 4, window=window, seed=3)


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 6, 2], [40, 90, 2]])
def test_peaked_scores(new):
    """Large queries: a few keys take all the weight, and the running maximum moves far."""
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 32, [700, 90, 2], seed=5)
    check(pool, new, q4.BF16, 8, spread=12.0, seed=5)


@pytest.mark.parametrize("new", [[1, 1], [40, 90]])
@pytest.mark.parametrize("fmt", FMTS)
def test_values_of_any_size(fmt, new):
    """Scales from 2^-10 to 2^10 within a cache: no operand overflows, none is lost."""
    pool = Pool(fmt, 32, 64, 1, 16, [333, 90], seed=8)
    rng = np.random.default_rng(9)
    for half in (1,):
        for b, n in enumerate(pool.lens):
            codes, scales, zeros, _ = pool.rows[half][b]
            scales *= np.exp2(rng.integers(-10, 11, (n, 1, 1))).astype(scales.dtype)
            from _kv import row_values
            pool.rows[half][b] = (codes, scales, zeros, row_values(fmt, 32, codes, scales, zeros))
            t = np.arange(n)
            pg, sl = torch.from_numpy(pool.table[b][t // 16]).to(DEV), torch.from_numpy(t % 16).to(DEV)
            pool.cache.v_scales[pg, :, sl] = torch.from_numpy(scales).to(DEV)
    check(pool, new, q4.F16 if fmt == q4.NF4 else q4.BF16, 2, seed=8)


@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
def test_queries_of_any_size(act):
    """Rows of tiny and of large queries (and one of zeros) beside each other."""
    pool = Pool(q4.INT4_ASYM, 64, 128, 1, 32, [260], seed=3)
    rng = np.random.default_rng(4)
    size = np.array([2.0 ** -13, 1.0, 0.0, 2.0 ** 9] + [2.0 ** e for e in range(-6, 6)])
    q = torch.from_numpy(rng.standard_normal((1, 16, 128)) * size[:, None]).to(DEV).to(TORCH[act])
    lse = torch.empty((1, 16), device=DEV)
    out = kv.attention(pool.cache, pool.batch(), q, scale=2.0 ** -8, lse=lse)
    ref, mag, rl, _, worst = attention_ref(pool, [1], q.double().cpu().numpy(), 2.0 ** -8)
    # each row by its own scores
    per_row = np.array([(np.abs(q[0, j].double().cpu().numpy()) @ np.abs(pool.values(0, 0)[:, 0]).T).max() for j in range(16)]) * 2.0 ** -8
    delta = (2.0 ** -24 * 144 * per_row + 2.0 ** -20)[None, :]
    assert (np.abs(lse.double().cpu().numpy() - rl) <= delta + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl)).all()
    tol = (2 * delta[..., None] + 2.0 ** -18 + 2.0 ** -10) * mag + UNIT[act] * np.abs(ref) + 260 * 2.0 ** -21 * 0.3
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("new", [[1, 1], [9, 4], [200, 100]])
def test_pages_that_do_not_exist(new):
    """Tokens whose page number is outside the pool take no part."""
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 16, [250, 120], seed=6)
    hidden = [np.zeros(n, dtype=bool) for n in pool.lens]
    for b, p, bad in ((0, 3, -1), (0, 4, 10 ** 9), (1, 0, -5)):
        pool.table[b, p] = bad
        hidden[b][16 * p:16 * p + 16] = True
    out, lse, md = check(pool, new, q4.BF16, 4, hidden=hidden, seed=3)


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 2, 2], [50, 60, 70]])
def test_every_row_empty(new):
    """Sequences of no cached token: zero outputs, -inf statistics, mass as it was."""
    pool = Pool(q4.NF4, 32, 64, 2, 16, [0, 0, 0], seed=6)
    check(pool, new, q4.F16, 8)


def test_long_split():
    """One long sequence beside short ones: the length is split, the parts joined."""
    pool = Pool(q4.INT4_ASYM, 64, 128, 1, 128, [20011, 3, 700], seed=12)
    check(pool, [1, 1, 1], q4.BF16, 4, seed=2)
    check(pool, [3, 3, 3], q4.BF16, 4, seed=3)
    check(pool, [1, 1, 1], q4.BF16, 4, window=9000, seed=4)


def test_chunk_on_long():
    pool = Pool(q4.INT4_SYM, 32, 64, 1, 64, [9001], seed=13)
    check(pool, [70], q4.F16, 2, seed=2)
    check(pool, [70], q4.F16, 2, window=3001, seed=2)


def test_loose_bounds():
    """max_len and max_new far above what the batch holds."""
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 32, [100, 40], seed=3, width=64)
    check(pool, [1, 1], q4.BF16, 8, batch=pool.batch())
    check(pool, [3, 2], q4.BF16, 8, batch=pool.batch([3, 2], max_new=500))
    check(pool, [3, 2], q4.BF16, 8, batch=pool.batch([3, 2], max_len=100))


def test_same_bits_every_time():
    pool = Pool(q4.INT4_SYM, 64, 128, 4, 64, [3000, 1500, 77], seed=3)
    for new in ([1, 1, 1], [4, 3, 2], [300, 200, 77]):
        first = check(pool, new, q4.BF16, 16, seed=1)
        again = check(pool, new, q4.BF16, 16, seed=1)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows more than 4 GiB into the pool."""
    pages = 5 * 2 ** 30 // (64 * 64 * 8)
    pool = Pool(q4.INT4_SYM, 64, 128, 8, 64, [200, 130], seed=3, pages=pages, first_page=pages - 9)
    check(pool, [1, 1], q4.BF16, 16)
    check(pool, [80, 130], q4.BF16, 16)


def test_graph_and_stream():
    """A decode step captured on a side stream, replayed as the sequences grow."""
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 32, [90, 300], seed=3, spare=4)
    rng = np.random.default_rng(3)
    q, qd = queries(rng, 2, 8, 128, q4.BF16)
    batch = pool.batch()
    lens = batch.lens
    mass = torch.zeros((2, 2, pool.table.shape[1] * 32), device=DEV)
    work = torch.empty((kv.workspace_bytes(pool.cache, batch, 8, True),), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.attention(pool.cache, batch, q, mass=mass, workspace=work)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = kv.attention(pool.cache, batch, q, mass=mass, workspace=work)
    for n in ([90, 300], [64, 299], [1, 2], [90, 17]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        mass.zero_()
        work.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        m2 = torch.zeros_like(mass)
        want = kv.attention(pool.cache, batch, q, mass=m2)
        assert torch.equal(out, want) and torch.equal(mass, m2)
        torch.cuda.synchronize()


def test_refusals():
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 32, [90, 30], seed=3)
    b = pool.batch()
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        kv.attention(pool.cache, b, q[:1])
    with pytest.raises(ValueError):
        kv.attention(pool.cache, b, q[..., :64])
    with pytest.raises(TypeError):
        kv.attention(pool.cache, b, q.float())
    with pytest.raises(q4.Q4Error):
        kv.attention(pool.cache, b, torch.zeros((2, 3, 128), dtype=torch.bfloat16, device=DEV))   # 3 heads over 2
    with pytest.raises(q4.Q4Error):
        kv.attention(pool.cache, b, q, scale=-1.0)
    with pytest.raises(q4.Q4Error):
        kv.attention(pool.cache, b, q, window=-1)
    with pytest.raises(q4.Q4Error):
        kv.attention(pool.cache, b, q, mass=torch.zeros((2, 2, 5), device=DEV))
    with pytest.raises(ValueError):
        kv.attention(pool.cache, b, q, mass=torch.zeros((2, 4, 500), device=DEV))
    for odd in (torch.zeros((2, 4, 132), dtype=torch.bfloat16, device=DEV)[..., :128],      # rows 264 bytes apart
                torch.zeros((2, 4, 136), dtype=torch.bfloat16, device=DEV)[..., 1:129]):    # and 2 bytes off
        with pytest.raises(q4.Q4Error):
            kv.attention(pool.cache, b, odd)
    with pytest.raises(q4.Q4Error):
        kv.attention(pool.cache, b, q, mass=torch.zeros((2, 2, 500), device=DEV),
                     workspace=torch.empty((1,), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        kv.Batch(b.table, b.lens, tokens=3)
    with pytest.raises(ValueError):
        kv.Batch(b.table, b.lens, torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        kv.Batch(b.table.long(), b.lens)
