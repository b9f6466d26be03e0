"""Windows wider than a C int, from Python: no limit, not their low 32 bits."""

import pytest
import torch

from bit_group_wise_amd import kv, q4
from test_kv_batch_cpu import Fake, ints, make_cache


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 64, 2 ** 40 + 1])
def test_wide_windows_are_no_limit(window):
    """16384 tokens take more parts, and so more workspace, than the 64 that a window of 64 leaves."""
    cache = make_cache(16)
    b = kv.Batch(ints(3, 1024), ints(3))
    size = lambda w: kv.workspace_bytes(cache, b, 4, window=w)  # noqa: E731
    assert size(64) < size(0) == size(16384) == size(window)


@pytest.mark.parametrize("window", [-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32 + 64])
def test_negative_windows_are_refused(window, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    cache = make_cache(16)
    b = kv.Batch(ints(3, 1024), ints(3))

    q, out = (Fake((3, 4, 64), torch.float16, 0x900000) for _ in range(2))
    work = Fake((1 << 20,), torch.uint8, 0xa00000)
    work.numel = lambda: 1 << 20
    with pytest.raises(q4.Q4Error) as e:   # (before anything is launched)
        kv.attention(cache, b, q, window=window, out=out, workspace=work)
    assert e.value.status == q4.EINVAL
