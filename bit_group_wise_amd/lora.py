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


def _tensor(t, name, dtype, shape, device):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


class Adapters:
    """Pairs a [n, rank, K] and b [n, N, rank] of one 16-bit type, and their
    scales, float32 [n] (None: 1)."""

    def __init__(self, a, b, scale=None):
        torch = _torch()
        if a.dim() != 3 or b.dim() != 3 or b.shape[0] != a.shape[0] or b.shape[2] != a.shape[1]:
            raise ValueError("a must be [adapters, rank, K] and b [adapters, N, rank]")
        _act_code(a.dtype)
        self.adapters, self.rank, self.K = a.shape
        self.N = b.shape[1]
        _tensor(a, "a", a.dtype, a.shape, a.device)
        _tensor(b, "b", a.dtype, b.shape, a.device)
        if scale is not None:
            _tensor(scale, "scale", torch.float32, (self.adapters,), a.device)
        self.a, self.b, self.scale = a, b, scale
        self.dtype, self.device = a.dtype, a.device

    def _record(self, x, q, ids, M, name):
        """The C record of a call on M rows, checked against the weight and the activations."""
        if (q.N, q.K) != (self.N, self.K) or q.codes.device != self.device:
            raise ValueError(f"the adapters are of a [{self.N}, {self.K}] weight on {self.device}")
        if x.dtype != self.dtype:
            raise TypeError(f"{name} must be {self.dtype}, as the adapters are, got {x.dtype}")
        ids_p = None if ids is None else _tensor(ids, "ids", _torch().int32, (M,), self.device)
        return _LoraArgs(self.a.data_ptr(), self.b.data_ptr(), q4._ptr(self.scale), ids_p, self.adapters, self.rank)


def _rows(t, name, width):
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError(f"{name} must be [rows, {width}], got {list(t.shape)}")
    return t.shape[0]


def workspace_bytes(M, pairs, backward=False) -> int:
    """Bytes of device workspace that a call on M rows needs (q4_lora_workspace_bytes)."""
    return lib().q4_lora_workspace_bytes(M, pairs.N, pairs.K, pairs.adapters, pairs.rank, int(backward))


def _workspace(workspace, M, pairs, backward):
    torch = _torch()
    if workspace is None:
        workspace = torch.empty((workspace_bytes(M, pairs, backward),), dtype=torch.uint8, device=pairs.device)
    else:
        _tensor(workspace, "workspace", torch.uint8, (workspace.numel(),), pairs.device)
    return workspace


def gemm(x, q, pairs, ids=None, *, out=None, workspace=None):
    """y = x . What^T + scale (x a^T) b^T with each row's adapter (q4_lora_gemm).
    workspace: a uint8 tensor of at least workspace_bytes, else one is
    allocated."""
    M = _rows(x, "x", pairs.K)
    rec = pairs._record(x, q, ids, M, "x")
    xp = _tensor(x, "x", x.dtype, x.shape, pairs.device)
    if out is None:
        out = x.new_empty((M, pairs.N))
    else:
        _tensor(out, "out", x.dtype, (M, pairs.N), pairs.device)
    work = _workspace(workspace, M, pairs, False)
    st = _launch(pairs.device, lib().q4_lora_gemm, q.fmt, q.g, _act_code(x.dtype), xp, M, q.codes.data_ptr(),
                 q.scales.data_ptr(), q4._ptr(q.zeros), q.N, q.K, ctypes.addressof(rec), out.data_ptr(),
                 work.data_ptr(), work.numel())
    _check(st, "q4_lora_gemm")
    return out


def backward(dy, x, q, pairs, ids=None, *, need_dx=True, need_pairs=True, out=None, workspace=None):
    """Gradients of gemm (q4_lora_backward): (dx [M, K], da, db), those not
    needed None (x may be None where the adapters' are not).  out: a tuple of
    three tensors to write, None where one is to be allocated."""
    M = _rows(dy, "dy", pairs.N)
    rec = pairs._record(dy, q, ids, M, "dy")
    dev = pairs.device
    dyp = _tensor(dy, "dy", dy.dtype, dy.shape, dev)
    if need_pairs or x is not None:
        xp = _tensor(x, "x", dy.dtype, (M, pairs.K), dev)
    else:
        xp = None
    got = []
    for t, name, shape, need in zip(out or (None,) * 3, ("dx", "da", "db"),
                                    ((M, pairs.K), pairs.a.shape, pairs.b.shape),
                                    (need_dx, need_pairs, need_pairs)):
        if not need:
            t = None
        elif t is None:
            t = dy.new_empty(shape)
        else:
            _tensor(t, name, dy.dtype, shape, dev)
        got.append(t)
    work = _workspace(workspace, M, pairs, True)
    st = _launch(dev, lib().q4_lora_backward, q.fmt, q.g, _act_code(dy.dtype), dyp, xp, M, q.codes.data_ptr(),
                 q.scales.data_ptr(), q4._ptr(q.zeros), q.N, q.K, ctypes.addressof(rec),
                 *(None if t is None else t.data_ptr() for t in got), work.data_ptr(), work.numel())
    _check(st, "q4_lora_backward")
    return tuple(got)
