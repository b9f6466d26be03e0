"""Windows that no sequence outgrows, up to the largest int, are no limit: the
same bits as without one, where sequences have more new tokens than cached ones too."""

import numpy as np
import pytest
import torch

from bit_group_wise_amd import kv, q4
from _kv import DEV, TORCH, Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new", [([90, 700], [1, 1]), ([90, 40, 0, 2], [3, 4, 1, 4]), ([3, 70, 200, 0], [9, 70, 37, 8]),
                                      ([1300, 20], [150, 80]), ([0, 0], [1, 1])])
@pytest.mark.parametrize("fmt", [q4.INT4_ASYM, q4.NF4])
def test_no_limit(fmt, lens, new):
    pool = Pool(fmt, 64, 128, 2, 16, lens, seed=len(lens))
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((sum(new), 4, 128))).to(DEV).to(TORCH[q4.BF16])
    batch = pool.batch(None if all(m == 1 for m in new) else new)
    width = pool.table.shape[1] * 16

    def call(window):
        mass = torch.ones((len(lens), 2, width), device=DEV)
        lse = torch.empty((sum(new), 4), device=DEV)
        return kv.attention(pool.cache, batch, q, window=window, mass=mass, lse=lse), lse, mass

    want = call(0)
    assert any(bool(t.isfinite().any()) for t in want)
    for window in (width, width + 1, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 32 + 64):
        print("window", window, flush=True)
        for a, b in zip(want, call(window)):
            assert torch.equal(a, b)
