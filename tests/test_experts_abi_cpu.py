"""Host-side checks of the experts' entry points that need no GPU: every bad
argument comes back as its documented status before any HIP call."""

import pytest

from bit_group_wise_amd import q4

A = 0x10000


def gemm(**kw):
    a = dict(f=q4.NF4, g=64, t=q4.BF16, x=A, xrows=4, index=None, offsets=A, rows=4, experts=2, codes=A, scales=A,
             zeros=None, N=64, K=128, y=A)
    a.update(kw)
    return q4.lib().q4_experts_gemm(*a.values(), None)


def dx(**kw):
    a = dict(f=q4.NF4, g=64, t=q4.BF16, dy=A, offsets=A, rows=4, experts=2, codes=A, scales=A, zeros=None, N=64,
             K=128, dx=A)
    a.update(kw)
    return q4.lib().q4_experts_gemm_dx(*a.values(), None)


BOTH = [
    (dict(f=9), q4.EUNSUPPORTED), (dict(g=48), q4.EUNSUPPORTED), (dict(t=2), q4.EUNSUPPORTED),
    (dict(codes=None), q4.EINVAL), (dict(scales=None), q4.EINVAL), (dict(offsets=None), q4.EINVAL),
    (dict(zeros=A), q4.EINVAL), (dict(f=q4.INT4_ASYM), q4.EINVAL),
    (dict(N=0), q4.EINVAL), (dict(N=-8), q4.EINVAL), (dict(K=0), q4.EINVAL), (dict(K=100), q4.EINVAL),
    (dict(experts=0), q4.EINVAL), (dict(experts=-1), q4.EINVAL), (dict(rows=-1), q4.EINVAL),
    (dict(experts=65537), q4.EUNSUPPORTED), (dict(N=2 ** 31), q4.EUNSUPPORTED), (dict(N=2 ** 62), q4.EUNSUPPORTED),
    (dict(experts=65536, N=32768), q4.EUNSUPPORTED),
    (dict(K=64 * 65537), q4.EUNSUPPORTED),
    (dict(codes=A + 8), q4.EALIGN), (dict(scales=A + 2), q4.EALIGN), (dict(offsets=A + 2), q4.EALIGN),
]


@pytest.mark.parametrize("kw,status", BOTH)
def test_both_refuse(kw, status):
    assert gemm(**kw) == status
    assert dx(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), q4.EINVAL), (dict(y=None), q4.EINVAL), (dict(xrows=3), q4.EINVAL), (dict(xrows=-1), q4.EINVAL),
    (dict(index=A, xrows=0), q4.EINVAL), (dict(x=A + 8), q4.EALIGN), (dict(y=A + 1), q4.EALIGN),
    (dict(index=A + 1), q4.EALIGN), (dict(index=A, xrows=2 ** 31 // 256), q4.EUNSUPPORTED),
    (dict(rows=2 ** 30 + 1, xrows=2 ** 30 + 1), q4.EUNSUPPORTED), (dict(rows=2 ** 62, xrows=2 ** 62), q4.EUNSUPPORTED),
    (dict(rows=2 ** 30, xrows=2 ** 30, N=4096), q4.EUNSUPPORTED),  # more workgroups than a grid has
])
def test_gemm_refuses(kw, status):
    assert gemm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), q4.EINVAL), (dict(dx=None), q4.EINVAL), (dict(N=60), q4.EUNSUPPORTED),
    (dict(dy=A + 8), q4.EALIGN), (dict(dx=A + 8), q4.EALIGN),
    (dict(N=8 * 524288, experts=1), q4.EUNSUPPORTED), (dict(N=262144, K=16384), q4.EUNSUPPORTED),
    (dict(N=8, K=64 * 16384, rows=2 ** 30, experts=1), q4.EUNSUPPORTED),  # more workgroups than a grid has
])
def test_dx_refuses(kw, status):
    assert dx(**kw) == status


def test_no_rows_is_no_work():
    assert gemm(rows=0, xrows=0, x=None, y=None) == q4.OK
    assert gemm(rows=0, index=A, x=None, y=None) == q4.OK
    assert dx(rows=0, dy=None, dx=None) == q4.OK
    assert gemm(rows=0, offsets=None) == q4.EINVAL
