"""Host-side checks of the key/value cache's C ABI that need no GPU: every bad
argument comes back as its documented status before any HIP call."""

import ctypes
import math

import pytest

from bit_group_wise_amd import kv, q4

A, MIS = 0x10000, 0x10002


def cache(**kw):
    a = dict(k_codes=A, k_scales=A, k_zeros=None, v_codes=A, v_scales=A, v_zeros=None, pages=8, page=16, heads=2,
             dim=128, g=64, format=q4.INT4_SYM, reserved=0)
    a.update(kw)
    return kv._CacheArgs(**a)


def batch(**kw):
    a = dict(table=A, lens=A, starts=None, tokens=3, table_width=4, seqs=3, max_new=1, max_len=64)
    a.update(kw)
    return kv._BatchArgs(**a)


def call_append(c=None, b=None, **kw):
    a = dict(t=q4.BF16, k=A, kts=256, khs=128, v=A, vts=256, vhs=128)
    a.update(kw)
    c, b = c or cache(), b or batch()
    return q4.lib().q4_kv_append(ctypes.addressof(c), ctypes.addressof(b), *a.values(), None)


def call_attention(c=None, b=None, **kw):
    a = dict(t=q4.BF16, q=A, qts=512, qhs=128, heads=4, scale=0.1, window=0, out=A, lse=None, mass=None, width=0,
             work=A, work_bytes=1 << 40)
    a.update(kw)
    c, b = c or cache(), b or batch()
    return q4.lib().q4_kv_attention(ctypes.addressof(c), ctypes.addressof(b), *a.values(), None)


def call_evict(c=None, b=None, **kw):
    a = dict(mass=A, width=64, table=A, tw=4, budget=32, recent=8, lens=A, nmass=A, nwidth=32, kept=A)
    a.update(kw)
    c, b = c or cache(), b or batch()
    return q4.lib().q4_kv_evict(ctypes.addressof(c), ctypes.addressof(b), *a.values(), None)


def call_read(c=None, b=None, t=q4.F16, k=A, v=A):
    c, b = c or cache(), b or batch()
    return q4.lib().q4_kv_read(ctypes.addressof(c), ctypes.addressof(b), t, k, v, None)


def test_record_layout():
    assert ctypes.sizeof(kv._CacheArgs) == 80 and kv._CacheArgs.pages.offset == 48
    assert ctypes.sizeof(kv._BatchArgs) == 48 and kv._BatchArgs.tokens.offset == 24


@pytest.mark.parametrize("call", [call_append, call_read, call_attention, call_evict])
@pytest.mark.parametrize("kw,status", [
    (dict(format=q4.NF4_DQ), q4.EUNSUPPORTED),
    (dict(format=9), q4.EUNSUPPORTED),
    (dict(g=16), q4.EUNSUPPORTED),
    (dict(dim=96, g=32), q4.EUNSUPPORTED),
    (dict(dim=64, g=128), q4.EINVAL),
    (dict(page=24), q4.EUNSUPPORTED),
    (dict(page=512), q4.EUNSUPPORTED),
    (dict(pages=0), q4.EINVAL),
    (dict(pages=2 ** 31), q4.EUNSUPPORTED),
    (dict(heads=0), q4.EINVAL),
    (dict(reserved=1), q4.EINVAL),
    (dict(k_codes=None), q4.EINVAL),
    (dict(v_scales=None), q4.EINVAL),
    (dict(k_zeros=A), q4.EINVAL),
    (dict(format=q4.INT4_ASYM), q4.EINVAL),
    (dict(format=q4.INT4_ASYM, k_zeros=A), q4.EINVAL),
    (dict(format=q4.INT4_ASYM, k_zeros=A, v_zeros=MIS), q4.EALIGN),
    (dict(v_codes=0x10008), q4.EALIGN),
    (dict(k_scales=0x10008), q4.EALIGN),
])
def test_cache_rejected(call, kw, status):
    assert call(c=cache(**kw)) == status


@pytest.mark.parametrize("call", [call_append, call_read, call_attention, call_evict])
@pytest.mark.parametrize("kw,status", [
    (dict(table=None), q4.EINVAL),
    (dict(lens=None), q4.EINVAL),
    (dict(seqs=0), q4.EINVAL),
    (dict(table_width=0), q4.EINVAL),
    (dict(max_len=-1), q4.EINVAL),
    (dict(max_len=65), q4.EINVAL),                       # more than the table can hold
    (dict(seqs=65536, tokens=65536), q4.EUNSUPPORTED),
    (dict(table_width=2 ** 30, max_len=2 ** 23), q4.EUNSUPPORTED),
    (dict(table=MIS), q4.EALIGN),
    (dict(lens=MIS), q4.EALIGN),
])
def test_batch_rejected(call, kw, status):
    assert call(b=batch(**kw)) == status


@pytest.mark.parametrize("call", [call_append, call_read, call_attention])
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=2), q4.EINVAL),                         # one a sequence without starts
    (dict(max_new=2), q4.EINVAL),
    (dict(tokens=-1, starts=A), q4.EINVAL),
    (dict(max_new=-1, starts=A), q4.EINVAL),
    (dict(tokens=2 ** 31, starts=A), q4.EUNSUPPORTED),
    (dict(starts=MIS), q4.EALIGN),
])
def test_rows_rejected(call, kw, status):
    assert call(b=batch(**kw)) == status


@pytest.mark.parametrize("call", [call_append, call_read, call_attention])
def test_nothing_to_do(call):
    assert call(b=batch(starts=A, tokens=0)) == q4.OK
    assert call(b=batch(starts=A, tokens=5, max_new=0)) == q4.OK


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), q4.EUNSUPPORTED),
    (dict(k=None), q4.EINVAL),
    (dict(v=None), q4.EINVAL),
    (dict(kts=-8), q4.EINVAL),
    (dict(k=0x10008), q4.EALIGN),
    (dict(khs=132), q4.EALIGN),
    (dict(vts=260), q4.EALIGN),
])
def test_append_rejected(kw, status):
    assert call_append(**kw) == status


@pytest.mark.parametrize("kw,status", [(dict(t=3), q4.EUNSUPPORTED), (dict(k=None), q4.EINVAL), (dict(v=0x10004), q4.EALIGN)])
def test_read_rejected(kw, status):
    assert call_read(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), q4.EUNSUPPORTED),
    (dict(heads=0), q4.EINVAL),
    (dict(heads=3), q4.EINVAL),
    (dict(heads=2 * 65), q4.EUNSUPPORTED),
    (dict(scale=0.0), q4.EINVAL),
    (dict(scale=-1.0), q4.EINVAL),
    (dict(scale=math.inf), q4.EINVAL),
    (dict(scale=math.nan), q4.EINVAL),
    (dict(window=-1), q4.EINVAL),
    (dict(q=None), q4.EINVAL),
    (dict(out=None), q4.EINVAL),
    (dict(qts=-8), q4.EINVAL),
    (dict(mass=A, width=63), q4.EINVAL),
    (dict(mass=A, width=64, work=None), q4.EINVAL),
    (dict(mass=A, width=64, work_bytes=4), q4.EINVAL),
    (dict(mass=A, width=64, work=0x10010), q4.EALIGN),
    (dict(q=0x10008), q4.EALIGN),
    (dict(out=0x10008), q4.EALIGN),
    (dict(qhs=100), q4.EALIGN),
    (dict(lse=MIS), q4.EALIGN),
    (dict(mass=MIS, width=64), q4.EALIGN),
])
def test_attention_rejected(kw, status):
    assert call_attention(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(mass=None), q4.EINVAL),
    (dict(table=None), q4.EINVAL),
    (dict(lens=None), q4.EINVAL),
    (dict(nmass=None), q4.EINVAL),
    (dict(kept=None), q4.EINVAL),
    (dict(budget=0), q4.EINVAL),
    (dict(recent=-1), q4.EINVAL),
    (dict(recent=33), q4.EINVAL),
    (dict(budget=65, nwidth=80), q4.EINVAL),             # more than new_table can hold
    (dict(width=63), q4.EINVAL),
    (dict(nwidth=31), q4.EINVAL),
    (dict(mass=MIS), q4.EALIGN),
    (dict(kept=MIS), q4.EALIGN),
])
def test_evict_rejected(kw, status):
    assert call_evict(**kw) == status


def test_workspace_bytes_of_bad_arguments():
    L = q4.lib()
    size = lambda c, b, h, m: L.q4_kv_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), h, 0, m)  # noqa: E731
    assert size(cache(g=16), batch(), 4, 1) == 0
    assert size(cache(), batch(seqs=0), 4, 1) == 0
    assert size(cache(), batch(), 3, 1) == 0
    assert size(cache(), batch(), 4, 1) > 0
