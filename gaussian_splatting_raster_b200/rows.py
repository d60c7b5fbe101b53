"""Per-row operators: scaled table lookup and feed-forward block, each with its gradient.

Thin binding of ``splat_lookup*`` and ``splat_ffn*`` (``include/splat.h``): checks tensors, takes
the scratch the library asks for from torch's allocator (on the stream the call runs on, so calls
on other streams and captured graphs have their own) and passes pointers. The calls write into the
caller's outputs, like the workspace's; nothing is recorded for autograd.

Row tensors may be views with any distance between rows (a column range of a wider tensor), their
columns contiguous. All tensors of a call have one type (fp32, bf16 or fp16) and one device.
"""
from __future__ import annotations

import torch

from . import SplatError, load_library

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_ACTS = {"silu": 0, "gelu": 1}
_MAX = 2**31 - 1  # the library's sizes are 32-bit


def _rows(t, name, like, shape):
    """Pointer and row distance (elements) of a [rows, cols] tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if max(shape) > _MAX:
        raise ValueError(f"{name} has a side of more than {_MAX}: {shape}")
    if t.numel() == 0:
        return None, shape[1]
    ld, step = t.stride()
    if shape[1] > 1 and step != 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _dense(t, name, like, shape):
    if t is None:
        return None
    p, ld = _rows(t, name, like, shape)
    if ld != shape[1]:
        raise ValueError(f"{name} must be contiguous")
    return p


def _first(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    return t


def _ids(ids, like):
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise TypeError("ids must be a CUDA tensor")
    if ids.dtype != torch.int32:
        raise TypeError(f"ids must be torch.int32, got {ids.dtype}")
    if ids.numel() > _MAX:
        raise ValueError(f"ids has more than {_MAX} entries")
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous vector")
    if ids.get_device() != like.get_device():
        raise ValueError(f"ids is on {ids.device}, expected {like.device}")
    return ids.data_ptr(), ids.shape[0]


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without an object


def _call(fn, what, t, stream, args, scratch_bytes=None):
    """fn(*args[, scratch, bytes], stream) on the device of tensor t; raises on a refusal."""
    dev = t.get_device()
    if stream is None and dev == torch.cuda.current_device():
        return _launch(fn, what, t, _raw_stream(dev), args, scratch_bytes)
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.device(dev):
        if stream is None:
            return _launch(fn, what, t, _raw_stream(dev), args, scratch_bytes)
        with torch.cuda.stream(stream):  # scratch belongs to the stream that uses it
            return _launch(fn, what, t, stream.cuda_stream, args, scratch_bytes)


def _launch(fn, what, t, stream, args, scratch_bytes):
    if scratch_bytes is not None:
        scratch = (torch.empty(scratch_bytes, dtype=torch.uint8, device=t.device)
                   if scratch_bytes else None)
        args = (*args, scratch.data_ptr() if scratch_bytes else None, scratch_bytes)
    rc = fn(*args, stream)
    if rc != 0:
        raise SplatError(rc, f"{what} refused its arguments" if rc in (-1, -2) else
                         f"{what} failed")


def lookup(table, ids, out, scale: float = 1.0, stream=None):
    """out[i] = scale * table[ids[i]]; a zero row where ids[i] is outside [0, N).
    table [N, C], ids [M] int32, out [M, C], C <= 8192."""
    _first(table, "table")
    N, C = table.shape
    pi, M = _ids(ids, table)
    pt, ldt = _rows(table, "table", table, (N, C))
    po, ldo = _rows(out, "out", table, (M, C))
    _call(load_library().splat_lookup, "lookup", table, stream,
          (pt, ldt, N, C, pi, M, scale, _DTYPES[table.dtype], po, ldo))


def lookup_backward(dout, ids, dtable, scale: float = 1.0, stream=None):
    """dtable[n] = scale * sum of dout[i] over ids[i] = n (every row is written).
    dout [M, C], ids [M] int32, dtable [N, C]."""
    _first(dout, "dout")
    M, C = dout.shape
    pi, n = _ids(ids, dout)
    if n != M:
        raise ValueError(f"ids has {n} entries, dout {M} rows")
    if not isinstance(dtable, torch.Tensor) or dtable.dim() != 2:
        raise TypeError("dtable must be a CUDA tensor of two dimensions")
    N = dtable.shape[0]
    pd, ldd = _rows(dout, "dout", dout, (M, C))
    pt, ldt = _rows(dtable, "dtable", dout, (N, C))
    L = load_library()
    _call(L.splat_lookup_backward, "lookup_backward", dout, stream,
          (pd, ldd, pi, M, C, scale, _DTYPES[dout.dtype], pt, ldt, N),
          L.splat_lookup_scratch(M, N, C))


def _weights(x, w_gate, w_up, w_down):
    _first(x, "x")
    _first(w_up, "w_up")
    _first(w_down, "w_down")
    M, D = x.shape
    F, O = w_up.shape[0], w_down.shape[0]
    return M, D, F, O, (_dense(w_gate, "w_gate", x, (F, D)), _dense(w_up, "w_up", x, (F, D)),
                        _dense(w_down, "w_down", x, (O, F)))


def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


def ffn(x, w_gate, w_up, w_down, y, act: str = "silu", stream=None):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T, or act(x w_up^T) w_down^T when w_gate is None.
    x [M, D], w_gate and w_up [F, D], w_down [O, F], y [M, O]; D, O <= 128, F <= 1024."""
    a = _act(act)
    M, D, F, O, w = _weights(x, w_gate, w_up, w_down)
    px, ldx = _rows(x, "x", x, (M, D))
    py, ldy = _rows(y, "y", x, (M, O))
    L, dt = load_library(), _DTYPES[x.dtype]
    _call(L.splat_ffn, "ffn", x, stream, (px, ldx, *w, py, ldy, M, D, F, O, dt, a),
          L.splat_ffn_scratch(M, D, F, O, dt, w_gate is not None, 0))


def ffn_backward(dy, x, w_gate, w_up, w_down, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                 act: str = "silu", stream=None):
    """Gradients of ffn from dy [M, O], each in its operand's shape; None leaves one out."""
    a = _act(act)
    M, D, F, O, w = _weights(x, w_gate, w_up, w_down)
    py, ldy = _rows(dy, "dy", x, (M, O))
    px, ldx = _rows(x, "x", x, (M, D))
    pd, ldd = (None, D) if dx is None else _rows(dx, "dx", x, (M, D))
    if dw_gate is not None and w_gate is None:
        raise ValueError("dw_gate needs w_gate")
    dw = (_dense(dw_gate, "dw_gate", x, (F, D)), _dense(dw_up, "dw_up", x, (F, D)),
          _dense(dw_down, "dw_down", x, (O, F)))
    if M == 0 and dx is not None and all(p is None for p in dw):
        return
    L, dt = load_library(), _DTYPES[x.dtype]
    _call(L.splat_ffn_backward, "ffn_backward", x, stream,
          (py, ldy, px, ldx, *w, pd, ldd, *dw, M, D, F, O, dt, a),
          L.splat_ffn_scratch(M, D, F, O, dt, w_gate is not None, 1))


def rows_status(stream=None):
    """Raise SplatError(DEVICE_TIMEOUT) when a bounded wait of these kernels ran out since the last
    call, on the stream's device (None: the current stream); waits for the stream."""
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):
        rc = load_library().splat_rows_status(s.cuda_stream)
    if rc != 0:
        raise SplatError(rc, "a bounded wait ran out" if rc == -6 else "reading the status failed")
