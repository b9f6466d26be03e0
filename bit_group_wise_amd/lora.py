"""Low-rank adapters beside a 4-bit weight (q4_lora_* of include/q4.h):
argument marshalling.

    pairs = lora.Adapters(a, b, scale)      # [n, rank, K], [n, N, rank], float32 [n]
    y = lora.gemm(x, q, pairs, ids)         # x [M, K]; ids int32 [M], -1: none
    dx, da, db = lora.backward(dy, x, q, pairs, ids)

Without ids every row has adapter 0.  The tensors are the caller's and may be
updated in place between calls (an optimiser's step on a and b).
"""

from __future__ import annotations

import ctypes

from . import q4
from .q4 import _act_code, _check, _launch, _torch, lib

_vp, _i32 = ctypes.c_void_p, ctypes.c_int32


class _LoraArgs(ctypes.Structure):
    _fields_ = [("a", _vp), ("b", _vp), ("scale", _vp), ("ids", _vp), ("adapters", _i32), ("rank", _i32)]


def _refuse(t, name, dtype, shape, index):
    """The error of a tensor that is not a contiguous CUDA one of this dtype and shape on this device."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")


def _tensor(t, name, dtype, shape, index):
    """t's address, if it is a contiguous CUDA tensor of this dtype and shape on this device."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, dtype, shape, index)
    return t.data_ptr()


class Adapters:
    """Pairs a [n, rank, K] and b [n, N, rank] of one 16-bit type, and their
    scales, float32 [n] (None: 1)."""

    def __init__(self, a, b, scale=None):
        torch = _torch()
        if a.dim() != 3 or b.dim() != 3 or b.shape[0] != a.shape[0] or b.shape[2] != a.shape[1]:
            raise ValueError("a must be [adapters, rank, K] and b [adapters, N, rank]")
        self._act = _act_code(a.dtype)
        self.adapters, self.rank, self.K = a.shape
        self.N = b.shape[1]
        self.dtype, self.device, self._index = a.dtype, a.device, a.get_device()
        args = [_tensor(a, "a", a.dtype, a.shape, self._index), _tensor(b, "b", a.dtype, b.shape, self._index), None]
        if scale is not None:
            args[2] = _tensor(scale, "scale", torch.float32, (self.adapters,), self._index)
        self.a, self.b, self.scale = a, b, scale
        self._int32 = torch.int32
        # what every call's record begins as, and the tensors as they were checked;
        # their storages are held, so that nothing else can come to lie at the
        # record's addresses
        self._args = _LoraArgs(*args, None, self.adapters, self.rank)
        self._checked = self._seen()
        self._held = tuple(t.untyped_storage() for t in (a, b, scale) if t is not None)
        self._sizes = {}

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"an Adapters' {name} cannot be replaced")
        super().__setattr__(name, value)

    def _seen(self):
        """Where the tensors lie and what they are now."""
        a, b, scale = self.a, self.b, self.scale
        if scale is None:
            return a.data_ptr(), b.data_ptr(), a.shape, b.shape, a.dtype, b.dtype
        return a.data_ptr(), b.data_ptr(), scale.data_ptr(), a.shape, b.shape, scale.shape, a.dtype, b.dtype, scale.dtype

    def _record(self, q, ids, M):
        """The C record of a call on M rows, to be held while it runs."""
        if q.N != self.N or q.K != self.K or q.codes.get_device() != self._index:
            raise ValueError(f"the adapters are of a [{self.N}, {self.K}] weight on {self.device}")
        if self._seen() != self._checked:
            # (storage or shape replaced in place, as by `.data =`, set_() or resize_())
            raise ValueError("the adapters' storage was replaced: make a new Adapters")
        if ids is None:
            return self._args
        rec = _LoraArgs.from_buffer_copy(self._args)
        rec.ids = _tensor(ids, "ids", self._int32, (M,), self._index)
        return rec

    def _bytes(self, M, backward):
        """q4_lora_workspace_bytes, asked once for each number of rows."""
        n = self._sizes.get((M, backward))
        if n is None:
            n = lib().q4_lora_workspace_bytes(M, self.N, self.K, self.adapters, self.rank, int(backward))
            if len(self._sizes) < 4096:
                self._sizes[M, backward] = n
        return n


def _rows(t, name, width, pairs):
    """Address and rows of a contiguous tensor [rows, width] of the adapters' type, on their device."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} must be [rows, {width}], got {list(shape)}")
    if t.dtype != pairs.dtype or t.get_device() != pairs._index or not t.is_contiguous():
        _refuse(t, name, pairs.dtype, shape, pairs._index)
    return t.data_ptr(), shape[0]


def workspace_bytes(M, pairs, backward=False) -> int:
    """Bytes of device workspace that a call on M rows needs (q4_lora_workspace_bytes);
    fewer rows may need more."""
    return pairs._bytes(M, bool(backward))


def _workspace(workspace, like, M, pairs, backward):
    """The workspace of a call, as the tensor given or a new one."""
    if workspace is None:
        return like.new_empty((pairs._bytes(M, backward),), dtype=_torch().uint8)
    _tensor(workspace, "workspace", _torch().uint8, (workspace.numel(),), pairs._index)
    return workspace


def gemm(x, q, pairs, ids=None, *, out=None, workspace=None):
    """y = x . What^T + scale (x a^T) b^T with each row's adapter (q4_lora_gemm).
    workspace: a uint8 tensor of at least workspace_bytes, else one is
    allocated."""
    xp, M = _rows(x, "x", pairs.K, pairs)
    rec = pairs._record(q, ids, M)
    if out is None:
        out = x.new_empty((M, pairs.N))
    else:
        _tensor(out, "out", pairs.dtype, (M, pairs.N), pairs._index)
    work = _workspace(workspace, x, M, pairs, False)
    zeros = q.zeros
    st = _launch(pairs.device, lib().q4_lora_gemm, q.fmt, q.g, pairs._act, xp, M, q.codes.data_ptr(),
                 q.scales.data_ptr(), None if zeros is None else zeros.data_ptr(), q.N, q.K, ctypes.addressof(rec),
                 out.data_ptr(), work.data_ptr(), work.numel())
    _check(st, "q4_lora_gemm")
    return out


def backward(dy, x, q, pairs, ids=None, *, need_dx=True, need_pairs=True, out=None, workspace=None):
    """Gradients of gemm (q4_lora_backward): (dx [M, K], da, db), those not
    needed None (x may be None where the adapters' are not).  out: a tuple of
    three tensors to write, None where one is to be allocated."""
    dyp, M = _rows(dy, "dy", pairs.N, pairs)
    rec = pairs._record(q, ids, M)
    index, dtype = pairs._index, pairs.dtype
    xp = None
    if need_pairs or x is not None:
        xp = _tensor(x, "x", dtype, (M, pairs.K), index)
    got = []
    for t, name, shape, need in zip(out or (None,) * 3, ("dx", "da", "db"),
                                    ((M, pairs.K), pairs.a.shape, pairs.b.shape),
                                    (need_dx, need_pairs, need_pairs)):
        if not need:
            t = None
        elif t is None:
            t = dy.new_empty(shape)
        else:
            _tensor(t, name, dtype, shape, index)
        got.append(t)
    work = _workspace(workspace, dy, M, pairs, True)
    st = _launch(pairs.device, lib().q4_lora_backward, q.fmt, q.g, pairs._act, dyp, xp, M, q.codes.data_ptr(),
                 q.scales.data_ptr(), q4._ptr(q.zeros), q.N, q.K, ctypes.addressof(rec),
                 *(None if t is None else t.data_ptr() for t in got), work.data_ptr(), work.numel())
    _check(st, "q4_lora_backward")
    return tuple(got)
