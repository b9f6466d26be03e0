"""A Batch and the records it hands to the C ABI, without a GPU: they outlive
the call that uses them, follow the batch's fields, and are made once for all
caches of a shape (a model has one cache a layer and one Batch a step)."""

import ctypes
import gc
import weakref

import pytest
import torch

from bit_group_wise_amd import kv, q4

DEVICE = torch.device("cuda:0")


class Fake:
    """What kv asks of a device tensor; its address is given."""

    def __init__(self, shape, dtype, ptr, device=DEVICE):
        self.shape, self.dtype, self.ptr, self.device = torch.Size(shape), dtype, ptr, device
        self.is_cuda = True

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return self.ptr

    def get_device(self):
        return self.device.index

    def stride(self):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)


def ints(*shape, ptr=0x1000, device=DEVICE):
    return Fake(shape, torch.int32, ptr, device)


def make_cache(page=16, heads=2, dim=64, at=0x100000, device=DEVICE, pages=8):
    half = lambda p: (Fake((pages, heads, page, dim // 2), torch.uint8, p, device),  # noqa: E731
                      Fake((pages, heads, page, dim // 64), torch.float16, p + 0x1000, device), None)
    return kv.KVCache(q4.INT4_SYM, 64, *half(at), *half(at + 0x8000))


class Library:
    """Stands in for libq4: keeps what a call was given, read at the time of the call and again after `meanwhile`."""

    def __init__(self):
        self.seen, self.asked, self.meanwhile = [], 0, None

    def read(self, addr):
        a = kv._BatchArgs.from_address(addr)
        return {n: getattr(a, n) for n, _ in a._fields_}

    def q4_kv_append(self, cache, batch, *rest):
        first = self.read(batch)
        if self.meanwhile is not None:
            self.meanwhile()
            gc.collect()
            junk = [kv._BatchArgs(*[1] * 8) for _ in range(50)]   # takes up what was freed
            assert self.read(batch) == first and junk
        self.seen.append(first)
        return q4.OK

    def q4_kv_workspace_bytes(self, cache, batch, heads, window, mass):
        self.asked += 1
        return 64



@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(kv, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return lib


def rows(batch, cache):
    return Fake((batch.tokens, cache.heads, cache.dim), torch.float16, 0x900000)


def append(cache, batch):
    x = rows(batch, cache)
    kv.append(cache, batch, x, x)


def test_records_do_not_replace_each_other(library):
    """Caches of two page sizes in turn: each call's record has its own bounds, and keeps them."""
    small, large = make_cache(16), make_cache(64)
    b = kv.Batch(ints(3, 4), ints(3, ptr=0x2000))
    for _ in range(3):
        append(small, b)
        append(large, b)
    assert [s["max_len"] for s in library.seen] == [64, 256] * 3


def test_record_lives_through_the_call(library):
    """What another thread does with the same batch during a call (the library releases Python's lock) leaves the call's record alone."""
    small, large = make_cache(16), make_cache(64)
    b = kv.Batch(ints(3, 4), ints(3, ptr=0x2000))

    def other_thread():
        library.meanwhile = None
        append(large, b)
        b.lens = ints(3, ptr=0x3000)
        append(large, b)
        append(small, b)

    library.meanwhile = other_thread
    append(small, b)
    assert [s["lens"] for s in library.seen] == [0x2000, 0x3000, 0x3000, 0x2000]


def test_assigned_fields_are_used(library):
    cache = make_cache(16)
    b = kv.Batch(ints(3, 4), ints(3, ptr=0x2000))
    append(cache, b)
    b.lens, b.table, b.max_len = ints(3, ptr=0x4000), ints(3, 9, ptr=0x5000), 77
    append(cache, b)
    assert (b.seqs, b.width) == (3, 9)
    b.starts, b.tokens, b.max_new = ints(4, ptr=0x6000), 11, 5
    append(cache, b)
    want = [dict(table=0x1000, lens=0x2000, starts=None, tokens=3, table_width=4, seqs=3, max_new=1, max_len=64),
            dict(table=0x5000, lens=0x4000, starts=None, tokens=3, table_width=9, seqs=3, max_new=1, max_len=77),
            dict(table=0x5000, lens=0x4000, starts=0x6000, tokens=11, table_width=9, seqs=3, max_new=5, max_len=77)]
    assert library.seen == want


def test_a_record_keeps_its_tensors():
    """The tensor that a record points to lives as long as a call may use the record."""
    cache, lens = make_cache(16), ints(3, ptr=0x2000)
    b = kv.Batch(ints(3, 4), lens)
    held = b._record(cache)
    alive = weakref.ref(lens)
    b.lens = ints(3, ptr=0x3000)
    del lens
    gc.collect()
    assert alive() is not None
    del held
    gc.collect()
    assert alive() is None


@pytest.mark.parametrize("field,value,error", [
    ("lens", ints(4), ValueError), ("lens", Fake((3,), torch.int64, 0x10), TypeError), ("table", ints(4, 4), ValueError),
    ("table", ints(12), ValueError), ("starts", ints(3), ValueError), ("tokens", 5, ValueError), ("max_new", 2, ValueError),
    ("lens", ints(3, device=torch.device("cuda:1")), ValueError)])
def test_assigned_fields_are_checked(library, field, value, error):
    cache = make_cache(16)
    b = kv.Batch(ints(3, 4), ints(3, ptr=0x2000))
    append(cache, b)
    setattr(b, field, value)
    with pytest.raises(error):
        kv.append(cache, b, Fake((3, 2, 64), torch.float16, 0x900000), Fake((3, 2, 64), torch.float16, 0x900000))
    assert len(library.seen) == 1


def test_other_device(library):
    b = kv.Batch(ints(3, 4), ints(3, ptr=0x2000))
    with pytest.raises(ValueError):
        append(make_cache(16, device=torch.device("cuda:1")), b)


def test_sizes_are_asked_once_for_a_shape(library):
    """Layers' caches of one shape share a record and its workspace sizes."""
    layers = [make_cache(16, at=0x100000 * (i + 1)) for i in range(4)]
    b = kv.Batch(ints(3, 4), ints(3, ptr=0x2000))
    for _ in range(3):
        for c in layers:
            assert kv.workspace_bytes(c, b, 4) == 64
    assert library.asked == 1
    kv.workspace_bytes(layers[0], b, 4, mass=True)
    kv.workspace_bytes(layers[1], b, 4, window=9)
    kv.workspace_bytes(layers[2], b, 8)
    kv.workspace_bytes(make_cache(16, heads=1), b, 4)
    assert library.asked == 5


def test_a_cache_keeps_its_tensors():
    """The library has a cache's addresses for good: its tensors cannot be exchanged."""
    c = make_cache(16)
    for name in ("k_codes", "v_scales", "page", "fmt"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))


@pytest.mark.parametrize("field", ["max_len", "max_new"])
@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5])
def test_bounds_past_32_bits_are_refused(field, n):
    """Not taken for their low 32 bits."""
    kw = dict(tokens=3, max_new=3)
    kw[field] = n
    with pytest.raises(ValueError):
        kv.Batch(ints(3, 4), ints(3), ints(4), **kw)


@pytest.mark.parametrize("budget,recent", [(8, 2 ** 32 + 3), (8, -2 ** 32 + 3), (2 ** 31, 0)])
def test_eviction_counts_past_32_bits_are_refused(library, monkeypatch, budget, recent):
    cache = make_cache(16)
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    mass, table = Fake((3, 2, 64), torch.float32, 0x10000), ints(3, 4)
    mass.new_empty = lambda shape: mass
    lens = ints(3)
    lens.new_empty = lambda shape: lens
    library.q4_kv_evict = lambda *a: pytest.fail("called")
    with pytest.raises(q4.Q4Error) as e:
        kv.evict(cache, kv.Batch(ints(3, 4), lens), mass, table, budget, recent)
    assert e.value.status == q4.EINVAL


@pytest.mark.parametrize("bad", ["address", "pages"])
def test_a_bad_cache_leaves_others_their_sizes(bad):
    """The library's answer of 0 for a cache that it refuses is not taken for another cache of the shape."""
    b = kv.Batch(ints(3, 1024), ints(3))
    good, other = make_cache(16), make_cache(16, at=0x100008 if bad == "address" else 0x100000, pages=0 if bad == "pages" else 8)
    assert kv.workspace_bytes(other, b, 4) == 0
    assert kv.workspace_bytes(good, b, 4) > 0
