"""The weights of a row sum to one: what all rows add to the mass is their number.

A row's weights are 2^(x - stat).  Its statistic is rounded to binary32, |stat| <
32 here, so its weights are off by at most ln 2 * 2^-20 together, by chance up or
down; over R rows the mean is off by 3 * 2^-20 ln 2 / sqrt(3 R) (three standard
deviations), and 2^-25 for sums that round: for the 512 rows and more of every
case less than 6e-8.  Summing 10^3 weights in binary32 adds chance errors alone.
The bound is 1.5e-7; half a last place of one sign would be 3e-7 and more."""

import numpy as np
import pytest
import torch

from bit_group_wise_amd import kv, q4
from _kv import DEV, FMTS, TORCH, Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new,heads,group", [
    ([700 + 13 * b for b in range(32)], None, 4, 4),          # single tokens, kept scores
    ([300 + 7 * b for b in range(32)], None, 2, 16),          # formed anew
    ([5000, 4000], [3, 3], 8, 16),                            # prompt kernel, split
    ([900, 400, 77], [900, 200, 77], 2, 2)])
@pytest.mark.parametrize("act", [q4.BF16, q4.F16])
@pytest.mark.parametrize("fmt", FMTS)
def test_total(fmt, act, lens, new, heads, group):
    pool = Pool(fmt, 64, 128, heads, 64, lens, seed=len(lens))
    tokens = len(lens) if new is None else sum(new)
    rng = np.random.default_rng(1)
    q = torch.from_numpy(rng.standard_normal((tokens, heads * group, 128)) * 1.5).to(DEV).to(TORCH[act])
    mass = torch.zeros((len(lens), heads, pool.table.shape[1] * 64), device=DEV)
    kv.attention(pool.cache, pool.batch(new), q, mass=mass)
    rows = tokens * heads * group
    assert rows >= 512
    assert abs(float(mass.double().sum()) / rows - 1) < 1.5e-7


def test_log_sum():
    """Against 64 bits: scores round by 2^-24 of their sum's size, the logarithm and its two parts by 2^-24 of 32."""
    lens = [2000, 900, 17]
    pool = Pool(q4.INT4_SYM, 64, 128, 2, 64, lens, seed=5)
    rng = np.random.default_rng(2)
    for new in ([1, 1, 1], [40, 30, 17]):
        q = torch.from_numpy(rng.standard_normal((sum(new), 32, 128))).to(DEV).bfloat16()
        lse = torch.empty((sum(new), 32), device=DEV)
        kv.attention(pool.cache, pool.batch(None if max(new) == 1 else new), q, lse=lse)
        got, qd, first, signed = lse.double().cpu().numpy(), q.double().cpu().numpy(), 0, []
        for b, (n, m) in enumerate(zip(lens, new)):
            see = np.arange(n) <= np.arange(n - m, n)[:, None]
            for j in range(32):
                x = qd[first:first + m, j] @ pool.values(0, b)[:, j // 16].T * float(np.float32(128 ** -0.5))
                want = np.log(np.where(see, np.exp(x), 0).sum(-1))
                signed.append(got[first:first + m, j] - want)
            first += m
        signed = np.concatenate(signed)
        assert np.abs(signed).max() < 4e-6 and abs(signed.mean()) < 3e-7
