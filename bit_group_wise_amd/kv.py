"""The 4-bit key/value cache (q4_kv_* of include/q4.h): argument marshalling.

A `KVCache` is the pool of pages, a `Batch` says which sequences a call works
on and where their new tokens are.  Both are thin handles over device tensors
that the caller owns and may update in place (lens, table) between calls; a
Batch's fields may also be assigned, and one Batch serves the caches of all
layers:

    cache = kv.alloc_cache(q4.INT4_SYM, 64, pages=512, page=64, heads=8, dim=128, device="cuda:0")
    step = kv.Batch(table, lens)                    # one new token a sequence
    kv.append(cache, step, k, v)                    # k, v [seqs, heads, dim]
    out = kv.attention(cache, step, q, mass=mass)   # q [seqs, q_heads, dim]
    lens, mass, kept = kv.evict(cache, step, mass, fresh_table, budget=1024, recent=128)

Prompts and drafts pass `starts`, the packed rows' offsets: sequence b's new
tokens are rows starts[b] .. starts[b+1] - 1 of k, v and q.
"""

from __future__ import annotations

import ctypes
import functools

from . import q4
from .q4 import _act_code, _check, _torch, lib

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _CacheArgs(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("k_zeros", _vp), ("v_codes", _vp),
                ("v_scales", _vp), ("v_zeros", _vp), ("pages", _i64), ("page", _i32), ("heads", _i32),
                ("dim", _i32), ("g", _i32), ("format", _i32), ("reserved", _i32)]


class _BatchArgs(ctypes.Structure):
    _fields_ = [("table", _vp), ("lens", _vp), ("starts", _vp), ("tokens", _i64),
                ("table_width", _i32), ("seqs", _i32), ("max_new", _i32), ("max_len", _i32)]


def _tensor(t, name, dtype, shape=None, device=None):
    """t as a contiguous CUDA tensor of this dtype and shape, or an error."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    return t


class KVCache:
    """Pages of 4-bit keys and values.

    codes uint8 [pages, heads, page, dim/2]; scales [pages, heads, page,
    dim/g], float16 (INT4) or float32 (NF4, FP4); zeros (INT4-asym) uint8
    [pages, heads, page, ceil(dim/g / 2)], else None."""

    def __init__(self, fmt, g, k_codes, k_scales, k_zeros, v_codes, v_scales, v_zeros):
        torch = _torch()
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, heads, page, dim/2]")
        pages, heads, page, half = k_codes.shape
        dim = 2 * half
        if fmt not in (q4.NF4, q4.INT4_SYM, q4.INT4_ASYM, q4.FP4):
            raise q4.Q4Error(q4.EUNSUPPORTED, "KVCache")
        if g not in (32, 64, 128):
            raise q4.Q4Error(q4.EUNSUPPORTED, "KVCache")
        if dim % g:
            raise q4.Q4Error(q4.EINVAL, "KVCache")
        sdt = torch.float32 if fmt in (q4.NF4, q4.FP4) else torch.float16
        dev, rows = k_codes.device, (pages, heads, page)
        for w, codes, scales, zeros in (("k", k_codes, k_scales, k_zeros), ("v", v_codes, v_scales, v_zeros)):
            _tensor(codes, w + "_codes", torch.uint8, (*rows, half), dev)
            _tensor(scales, w + "_scales", sdt, (*rows, dim // g), dev)
            if (fmt == q4.INT4_ASYM) != (zeros is not None):
                raise ValueError(w + "_zeros belong to INT4-asym caches, and to them alone")
            if zeros is not None:
                _tensor(zeros, w + "_zeros", torch.uint8, (*rows, (dim // g + 1) // 2), dev)
        self.fmt, self.g, self.pages, self.heads, self.page, self.dim = fmt, g, pages, heads, page, dim
        self.k_codes, self.k_scales, self.k_zeros = k_codes, k_scales, k_zeros
        self.v_codes, self.v_scales, self.v_zeros = v_codes, v_scales, v_zeros
        self.device, self._index = dev, dev.index
        # The current stream as the raw handle: a decode step makes a few calls
        # of some microseconds each, of which a stream object is one.
        self._stream = functools.partial(torch._C._cuda_getCurrentRawStream, dev.index)
        self._args = _CacheArgs(*(None if t is None else t.data_ptr() for t in
                                  (k_codes, k_scales, k_zeros, v_codes, v_scales, v_zeros)),
                                pages, page, heads, dim, g, fmt, 0)
        self._ref = ctypes.addressof(self._args)
        # What a batch's record and workspace sizes go by: all that the library
        # checks of a cache (it answers 0 for one that it refuses).
        self._key = (dev.index, fmt, g, pages, page, heads, dim,
                     all(t is None or t.data_ptr() % 16 == 0 for t in
                         (k_codes, k_scales, k_zeros, v_codes, v_scales, v_zeros)))

    def __setattr__(self, name, value):
        # (_args holds their addresses for good)
        if name in self.__dict__:
            raise AttributeError(f"a KVCache's {name} cannot be replaced")
        super().__setattr__(name, value)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.k_codes, self.k_scales, self.k_zeros, self.v_codes, self.v_scales, self.v_zeros)
                   if t is not None)


def alloc_cache(fmt, g, pages, page, heads, dim, device) -> KVCache:
    """A zeroed cache of `pages` pages."""
    torch = _torch()
    sdt = torch.float32 if fmt in (q4.NF4, q4.FP4) else torch.float16
    if g not in (32, 64, 128):
        raise q4.Q4Error(q4.EUNSUPPORTED, "alloc_cache")
    if dim <= 0 or dim % g:
        raise q4.Q4Error(q4.EINVAL, "alloc_cache")

    def half():
        z = lambda n, dt: torch.zeros((pages, heads, page, n), dtype=dt, device=device)  # noqa: E731
        return (z(dim // 2, torch.uint8), z(dim // g, sdt),
                z((dim // g + 1) // 2, torch.uint8) if fmt == q4.INT4_ASYM else None)

    return KVCache(fmt, g, *half(), *half())


class _Record:
    """What a call hands to C of a batch.  Whoever holds a record may use its
    address: it keeps the tensors that it points to, and nothing changes it."""

    __slots__ = ("args", "addr", "tensors", "sizes", "seqs", "tokens", "lens")

    def __init__(self, batch, page):
        table, lens, starts = batch.table, batch.lens, batch.starts
        self.seqs, width = table.shape
        self.tokens, self.lens, self.tensors = batch.tokens, lens, (table, starts)
        self.args = _BatchArgs(table.data_ptr(), lens.data_ptr(), None if starts is None else starts.data_ptr(),
                               batch.tokens, width, self.seqs, batch.max_new,
                               width * page if batch.max_len is None else batch.max_len)
        self.addr = ctypes.addressof(self.args)
        self.sizes = {}

    def workspace(self, cache, q_heads, window, mass):
        """q4_kv_workspace_bytes, asked once for each kind of call."""
        key = (q_heads, window, mass)
        n = self.sizes.get(key)
        if n is None:
            n = self.sizes[key] = lib().q4_kv_workspace_bytes(cache._ref, self.addr, q_heads, window, int(mass))
        return n


class Batch:
    """Sequences of a call: table int32 [seqs, width] of page numbers, lens
    int32 [seqs] (new tokens counted), and for more or fewer than one new token
    a sequence starts int32 [seqs + 1], the total `tokens` and the largest
    number `max_new`.  max_len bounds lens (default: what the table can hold);
    a tight bound spares work.  The fields may be assigned between calls; the
    next call checks them anew."""

    def __init__(self, table, lens, starts=None, *, tokens=None, max_new=None, max_len=None):
        if table.dim() != 2:
            raise ValueError("table must be [seqs, width]")
        if starts is None:
            tokens, max_new = table.shape[0] if tokens is None else tokens, 1 if max_new is None else max_new
        elif tokens is None or max_new is None:
            raise ValueError("starts needs tokens and max_new")
        self.table, self.lens, self.starts = table, lens, starts
        self.tokens, self.max_new, self.max_len = tokens, max_new, max_len
        self._check()

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        # records by KVCache._key, made of the fields as they are now; a call
        # that is under way keeps the one it has
        super().__setattr__("_records", {})

    @property
    def seqs(self):
        return self.table.shape[0]

    @property
    def width(self):
        return self.table.shape[1]

    @property
    def device(self):
        return self.table.device

    def _check(self):
        torch = _torch()
        if self.table.dim() != 2:
            raise ValueError("table must be [seqs, width]")
        _tensor(self.table, "table", torch.int32)
        _tensor(self.lens, "lens", torch.int32, (self.seqs,), self.device)
        if self.starts is not None:
            _tensor(self.starts, "starts", torch.int32, (self.seqs + 1,), self.device)
        elif self.tokens != self.seqs or self.max_new != 1:
            raise ValueError("without starts, every sequence has one new token")
        # (the record's fields are C ints, which would take the low 32 bits)
        for name in ("max_new", "max_len"):
            n = getattr(self, name)
            if n is not None and not -2 ** 31 <= n < 2 ** 31:
                raise ValueError(f"{name} must fit 32 bits, got {n}")

    def _record(self, cache):
        """The C record for caches of this one's shape (its page size bounds the
        lengths).  To be held while a call uses its address."""
        records = self._records
        rec = records.get(cache._key)
        if rec is None:
            self._check()
            if self.device != cache.device:
                raise ValueError(f"the batch is on {self.device}, the cache on {cache.device}")
            rec = records[cache._key] = _Record(self, cache.page)
        return rec


def _rows(t, name, tokens, heads, cache):
    """Checks of a packed [tokens, heads, dim] array (rows contiguous); its
    strides between tokens and heads (one over an axis of one says nothing)."""
    if t.shape != (tokens, heads, cache.dim):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {cache.dim}], got {list(t.shape)}")
    if t.get_device() != cache._index:  # (-1 on the host)
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return ts if tokens > 1 else 0, hs if heads > 1 else 0


def append(cache, batch, k, v):
    """Code the new tokens' keys and values [tokens, heads, dim] (fp16 or bf16,
    rows contiguous, any multiple of 8 between them) into their pages
    (q4_kv_append)."""
    rec = batch._record(cache)
    ks = _rows(k, "k", rec.tokens, cache.heads, cache)
    vs = _rows(v, "v", rec.tokens, cache.heads, cache)
    if v.dtype != k.dtype:
        raise TypeError("k and v must have one dtype")
    st = lib().q4_kv_append(cache._ref, rec.addr, _act_code(k.dtype), k.data_ptr(), *ks, v.data_ptr(), *vs,
                            cache._stream())
    _check(st, "q4_kv_append")


def read(cache, batch, dtype, out=None):
    """The new tokens' keys and values as the cache holds them, dequantized to
    [tokens, heads, dim] (q4_kv_read).  Returns (k, v)."""
    torch = _torch()
    rec = batch._record(cache)
    code = _act_code(dtype)
    shape = (rec.tokens, cache.heads, cache.dim)
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=cache.device)
        v = torch.empty_like(k)
    else:
        for t in out:
            _tensor(t, "out", dtype, shape, cache.device)
        k, v = out
    st = lib().q4_kv_read(cache._ref, rec.addr, code, k.data_ptr(), v.data_ptr(), cache._stream())
    _check(st, "q4_kv_read")
    return k, v


def _window(window):
    """A window as a C int: one past its range is no limit, as any that no sequence outgrows."""
    return window if -1 <= window <= 0x7fffffff else 0x7fffffff if window > 0 else -1


def workspace_bytes(cache, batch, q_heads, mass=False, window=0) -> int:
    """Bytes of device workspace that attention needs (q4_kv_workspace_bytes)."""
    return batch._record(cache).workspace(cache, q_heads, _window(window), bool(mass))


def attention(cache, batch, q, *, scale=None, window=0, mass=None, lse=None, out=None, workspace=None):
    """Attention of the new tokens' queries [tokens, q_heads, dim] over the
    cached tokens (q4_kv_attention).

    scale defaults to dim ** -0.5.  window > 0 lets a token see only the last
    `window` positions up to its own.  mass, float32 [seqs, heads, width >=
    max_len], gets each cached token's softmax weights added in place.  lse,
    float32 [tokens, q_heads], receives the log-sum-exp.  workspace: a uint8
    tensor of at least workspace_bytes, else one is allocated."""
    torch = _torch()
    rec = batch._record(cache)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, dim]")
    heads = q.shape[1]
    qs = _rows(q, "q", rec.tokens, heads, cache)
    code = _act_code(q.dtype)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _tensor(out, "out", q.dtype, (rec.tokens, heads, cache.dim), cache.device)
    mass_p, width = None, 0
    if mass is not None:
        if mass.dim() != 3:
            raise ValueError("mass must be [seqs, heads, width]")
        width = mass.shape[2]
        _tensor(mass, "mass", torch.float32, (rec.seqs, cache.heads, width), cache.device)
        mass_p = mass.data_ptr()
    lse_p = None
    if lse is not None:
        lse_p = _tensor(lse, "lse", torch.float32, (rec.tokens, heads), cache.device).data_ptr()
    window = _window(window)
    need = rec.workspace(cache, heads, window, mass is not None)
    work_p, have = None, 0
    if workspace is not None:
        _tensor(workspace, "workspace", torch.uint8, None, cache.device)
        work_p, have = workspace.data_ptr(), workspace.numel()
    elif need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=cache.device)
        work_p, have = workspace.data_ptr(), need
    st = lib().q4_kv_attention(cache._ref, rec.addr, code, q.data_ptr(), *qs, heads,
                               cache.dim ** -0.5 if scale is None else scale, window, out.data_ptr(), lse_p,
                               mass_p, width, work_p, have, cache._stream())
    _check(st, "q4_kv_attention")
    return out


def evict(cache, batch, mass, new_table, budget, recent, *, width=None):
    """Keep `budget` tokens of every sequence and head that has more: the last
    `recent` and the heaviest others by mass (q4_kv_evict; tokens on pages that
    do not exist neither stay nor count).  They move to the pages that
    new_table [seqs, new_width] names, free pages of this pool.  Returns
    (new_lens [seqs], new_mass [seqs, heads, width], kept [seqs, heads,
    budget]); width defaults to what new_table can hold."""
    torch = _torch()
    rec = batch._record(cache)
    if mass.dim() != 3:
        raise ValueError("mass must be [seqs, heads, width]")
    _tensor(mass, "mass", torch.float32, (rec.seqs, cache.heads, mass.shape[2]), cache.device)
    if new_table.dim() != 2:
        raise ValueError("new_table must be [seqs, width]")
    _tensor(new_table, "new_table", torch.int32, (rec.seqs, new_table.shape[1]), cache.device)
    if not 0 < budget < 2 ** 31 or not 0 <= recent <= budget:
        raise q4.Q4Error(q4.EINVAL, "q4_kv_evict")
    if width is None:
        width = new_table.shape[1] * cache.page
    new_lens = torch.empty_like(rec.lens)
    new_mass = mass.new_empty((rec.seqs, cache.heads, width))
    kept = new_lens.new_empty((rec.seqs, cache.heads, budget))
    st = lib().q4_kv_evict(cache._ref, rec.addr, mass.data_ptr(), mass.shape[2], new_table.data_ptr(),
                           new_table.shape[1], budget, recent, new_lens.data_ptr(), new_mass.data_ptr(),
                           width, kept.data_ptr(), cache._stream())
    _check(st, "q4_kv_evict")
    return new_lens, new_mass, kept
