"""fp16 outputs of attention over the 4-bit cache: of few rows they are off by
their own rounding alone, of many by that and the values' one rounding to fp16
(by none of it where a token's values have one scale).  Weights enter the
product in two fp16 parts (what is left is 2^-22 of a weight, less than the
2^-18 allowed for the scores)."""

import numpy as np
import pytest

from bit_group_wise_amd import q4
from _kv import FMTS, Pool
from test_gpu_kv_hidden import check, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("fmt", FMTS)
def test_few_rows(fmt, dim, g):
    """Single tokens, several, and as many rows as the few-row kernel takes."""
    most = (64 if dim == 64 else 32) // (dim // g)
    pool = Pool(fmt, g, dim, 2, 16, [140, 75, 41], seed=dim + g)
    for new, heads in (([1, 1, 1], 2), ([1, 1, 1], 2 * most), ([most, max(1, most - 1), 1], 2)):
        check(pool, new, q4.F16, queries(sum(new), heads, dim, q4.F16, 5), roundings=0)


def test_split():
    pool = Pool(q4.INT4_ASYM, 32, 128, 1, 32, [5000, 3, 700], seed=2)
    check(pool, [1, 1, 1], q4.F16, queries(3, 4, 128, q4.F16, 6), roundings=0)


@pytest.mark.parametrize("dim,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("fmt", FMTS)
def test_prompts(fmt, dim, g):
    """Each output within its bound; all together no further off than two equal
    and independent roundings, sqrt(2) of the output's own (2 % more for chance
    over some 10^5 outputs and for the scores)."""
    pool = Pool(fmt, g, dim, 2, 16, [300, 75], seed=dim + g)
    got, want = check(pool, [150, 75], q4.F16, queries(225, 4, dim, q4.F16, 5), roundings=0 if dim == g else 1)
    own = np.linalg.norm(want.astype(np.float16).astype(np.float64) - want)
    assert np.linalg.norm(got - want) <= (1.02 if dim == g else 1.45) * own
