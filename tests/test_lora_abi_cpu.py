"""Host-side checks of the adapters' entry points that need no GPU: every bad
argument comes back as its documented status before any HIP call."""

import ctypes

import pytest

from bit_group_wise_amd import lora, q4

A = 0x10000


def pairs(**kw):
    a = dict(a=A, b=A, scale=A, ids=A, adapters=2, rank=16)
    a.update(kw)
    return lora._LoraArgs(**a)


def gemm(rec=None, **kw):
    a = dict(f=q4.NF4, g=64, t=q4.BF16, x=A, M=4, codes=A, scales=A, zeros=None, N=64, K=128,
             low=ctypes.byref(rec or pairs()), y=A, work=A, bytes=1 << 40)
    a.update(kw)
    return q4.lib().q4_lora_gemm(*a.values(), None)


def backward(rec=None, **kw):
    a = dict(f=q4.NF4, g=64, t=q4.BF16, dy=A, x=A, M=4, codes=A, scales=A, zeros=None, N=64, K=128,
             low=ctypes.byref(rec or pairs()), dx=A, da=A, db=A, work=A, bytes=1 << 40)
    a.update(kw)
    return q4.lib().q4_lora_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(f=9), q4.EUNSUPPORTED), (dict(g=48), q4.EUNSUPPORTED), (dict(t=2), q4.EUNSUPPORTED),
    (dict(codes=None), q4.EINVAL), (dict(scales=None), q4.EINVAL), (dict(zeros=A), q4.EINVAL),
    (dict(f=q4.INT4_ASYM), q4.EINVAL), (dict(N=0), q4.EINVAL), (dict(K=0), q4.EINVAL), (dict(K=100), q4.EINVAL),
    (dict(M=-1), q4.EINVAL), (dict(M=2 ** 24 + 1), q4.EUNSUPPORTED), (dict(M=2 ** 62), q4.EUNSUPPORTED),
    (dict(N=2 ** 40), q4.EUNSUPPORTED), (dict(K=64 * 65537), q4.EUNSUPPORTED),
    (dict(low=None), q4.EINVAL), (dict(work=None), q4.EINVAL), (dict(bytes=0), q4.EINVAL),
    (dict(codes=A + 8), q4.EALIGN), (dict(scales=A + 2), q4.EALIGN), (dict(work=A + 128), q4.EALIGN),
    (dict(x=A + 8), q4.EALIGN),
])
def test_both_refuse(kw, status):
    assert gemm(**kw) == status and backward(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), q4.EINVAL), (dict(b=None), q4.EINVAL), (dict(adapters=0), q4.EINVAL), (dict(adapters=-1), q4.EINVAL),
    (dict(rank=0), q4.EINVAL), (dict(rank=-8), q4.EINVAL), (dict(rank=12), q4.EUNSUPPORTED),
    (dict(rank=264), q4.EUNSUPPORTED), (dict(adapters=16384), q4.EUNSUPPORTED),
    (dict(a=A + 8), q4.EALIGN), (dict(b=A + 8), q4.EALIGN), (dict(scale=A + 2), q4.EALIGN), (dict(ids=A + 2), q4.EALIGN),
])
def test_adapters_refused(kw, status):
    p = pairs(**kw)
    assert gemm(p) == status and backward(p) == status


@pytest.mark.parametrize("kw,status", [(dict(x=None), q4.EINVAL), (dict(y=None), q4.EINVAL), (dict(y=A + 1), q4.EALIGN)])
def test_gemm_refuses(kw, status):
    assert gemm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), q4.EINVAL), (dict(x=None), q4.EINVAL), (dict(da=None), q4.EINVAL), (dict(db=None), q4.EINVAL),
    (dict(dx=None, da=None, db=None), q4.EINVAL), (dict(N=60), q4.EUNSUPPORTED),
    (dict(dy=A + 8), q4.EALIGN), (dict(dx=A + 8), q4.EALIGN), (dict(da=A + 8), q4.EALIGN), (dict(db=A + 2), q4.EALIGN),
    (dict(N=262144, K=16384), q4.EUNSUPPORTED),
])
def test_backward_refuses(kw, status):
    assert backward(**kw) == status


def test_an_adapter_past_32_bits():
    assert gemm(pairs(rank=256), N=2 ** 22 + 8) == q4.EUNSUPPORTED
    assert gemm(pairs(rank=256), K=4194304, N=8) == q4.EUNSUPPORTED


def test_more_tiles_than_a_grid_has():
    assert gemm(M=2 ** 24, N=2 ** 20, K=64) == q4.EUNSUPPORTED
    assert backward(M=2 ** 24, N=8, K=2 ** 20) == q4.EUNSUPPORTED


def test_workspace_bytes():
    f = q4.lib().q4_lora_workspace_bytes
    assert f(0, 64, 64, 1, 8, 0) == 0 and f(4, 64, 64, 1, 12, 0) == 0 and f(-1, 64, 64, 1, 8, 1) == 0
    for M in (1, 16, 100, 5000):
        for rank in (8, 72, 256):
            fwd, bwd = f(M, 4096, 4096, 3, rank, 0), f(M, 4096, 4096, 3, rank, 1)
            # the parts' sums of outputs: at most 256 tiles of 64 x 128 binary32 values, for more than 96 rows
            sums = 256 * 64 * 128 * 4 if M > 96 else 0
            assert fwd % 256 == 0 and bwd % 256 == 0 and 4 * M * rank <= fwd <= 9 * 4 * M * rank + 512 + sums
            assert bwd > (fwd - sums) / 8
            assert gemm(pairs(adapters=3, rank=rank), M=M, N=4096, K=4096, bytes=fwd - 1) == q4.EINVAL
            assert backward(pairs(adapters=3, rank=rank), M=M, N=4096, K=4096, bytes=bwd - 1) == q4.EINVAL


def test_no_rows_is_no_work():
    assert gemm(M=0, x=None, y=None, work=None, bytes=0) == q4.OK


def test_the_gradient_of_no_rows():
    """An empty tensor's address may be NULL, whichever gradients are wanted."""
    none = dict(M=0, dy=None, x=None, da=None, db=None, work=None, bytes=0)
    assert backward(**none) == q4.OK and backward(dx=None, **none) == q4.OK
    assert backward(**dict(none, da=A)) == q4.EINVAL and backward(**dict(none, db=A)) == q4.EINVAL
    assert backward(pairs(rank=12), **none) == q4.EUNSUPPORTED and backward(**dict(none, dx=A + 8)) == q4.EALIGN
