"""Products through the 4-bit weights of a mixture's experts (q4_experts_* of
include/q4.h): argument marshalling.

The experts' weights are one QuantizedWeight of their stacked rows, and the
activations' rows are sorted by expert, `offsets` saying where each expert's
begin (int32 [experts + 1] on the device, as a cumulative count gives them):

    q = q4.quantize(weights.view(experts * N, K), q4.NF4, 64)   # [experts, N, K] fp16
    order = expert_of_row.argsort(stable=True)                  # rows: each token once per expert
    offsets = ...                                               # [experts + 1]
    y = experts.gemm(x, q, offsets, index=token_of_row[order])  # [rows, N]
    dx = experts.gemm_dx(dy, q, offsets)                        # [rows, K]
"""

from __future__ import annotations

from .q4 import _act_code, _check, _launch, _torch, lib


def _refuse(t, name, device):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, the weight on {device}")


def _rows(t, name, width, device):
    if t.get_device() != device.index or not t.is_contiguous():
        _refuse(t, name, device)
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} must be [rows, {width}], got {list(shape)}")
    return shape[0]


def _index(t, name, device):
    if t.get_device() != device.index or not t.is_contiguous():
        _refuse(t, name, device)
    if t.dtype != _torch().int32 or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D int32 tensor")
    return t.data_ptr()


def _groups(q, offsets, device):
    """Pointer of the offsets, experts and rows of each expert's weight."""
    p = _index(offsets, "offsets", device)
    experts = offsets.shape[0] - 1
    if experts < 1 or q.N % experts:
        raise ValueError(f"offsets must be [experts + 1], experts a divisor of the weight's {q.N} rows")
    return p, experts, q.N // experts


def _out(out, rows, width, like):
    if out is None:
        return like.new_empty((rows, width))
    if _rows(out, "out", width, like.device) != rows or out.dtype != like.dtype:
        raise ValueError(f"out must be {like.dtype} [{rows}, {width}]")
    return out


def gemm(x, q, offsets, *, index=None, out=None):
    """y[r] = x[index[r]] . What_e^T for the rows r of each expert e
    (q4_experts_gemm); x [tokens, K], index int32 [rows] (None: row r of x),
    offsets int32 [experts + 1].  Rows of `out` outside every group are left as
    they were."""
    dev = q.codes.device
    n = _rows(x, "x", q.K, dev)
    act = _act_code(x.dtype)
    off, experts, N = _groups(q, offsets, dev)
    rows, idx = n, None
    if index is not None:
        idx, rows = _index(index, "index", dev), index.shape[0]
    y = _out(out, rows, N, x)
    zeros = q.zeros
    st = _launch(dev, lib().q4_experts_gemm, q.fmt, q.g, act, x.data_ptr(), n, idx, off, rows, experts,
                 q.codes.data_ptr(), q.scales.data_ptr(), None if zeros is None else zeros.data_ptr(), N, q.K,
                 y.data_ptr())
    _check(st, "q4_experts_gemm")
    return y


def gemm_dx(dy, q, offsets, *, out=None):
    """dx[r] = dy[r] . What_e for the rows r of each expert e
    (q4_experts_gemm_dx); dy [rows, N].  The gradient of gathered rows is the
    sum of a token's rows of dx."""
    dev = q.codes.device
    off, experts, N = _groups(q, offsets, dev)
    rows = _rows(dy, "dy", N, dev)
    act = _act_code(dy.dtype)
    dx = _out(out, rows, q.K, dy)
    zeros = q.zeros
    st = _launch(dev, lib().q4_experts_gemm_dx, q.fmt, q.g, act, dy.data_ptr(), off, rows, experts,
                 q.codes.data_ptr(), q.scales.data_ptr(), None if zeros is None else zeros.data_ptr(), N, q.K,
                 dx.data_ptr())
    _check(st, "q4_experts_gemm_dx")
    return dx
