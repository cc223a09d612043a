"""Python binding of the post-training operators (``include/liger_train.h``).

As in ``_native``, every function has the name of the C entry point it calls,
takes torch tensors that already live on the GPU, runs on the current stream
and raises ``LigerError`` on a non-zero status.  What the library cannot see
(device, dtype, shape and contiguity of the tensors) is checked here and raises
``ValueError`` or ``TypeError``.
"""
from __future__ import annotations

import os
import re

from . import _native
from ._native import _F, _I64, _INT, _P, _SZ, LIGER_BF16, LIGER_F32, _check, _ptr, _stream

HEADER = os.path.join(os.path.dirname(_native.PKG), "include", "liger_train.h")

SIGNATURES = {
    "liger_block_norm_fwd": ([_P] * 9 + [_I64] * 3 + [_F] * 3 + [_INT, _P], _INT),
    "liger_block_norm_bwd_workspace": ([_I64] * 3, _SZ),
    "liger_block_norm_bwd": ([_P] * 15 + [_SZ] + [_I64] * 3 + [_F] * 2 + [_INT, _P], _INT),
}

_loaded = None


def header_functions() -> list:
    """Names of the functions include/liger_train.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(liger_[a-z_0-9]+)\s*\(", text, re.M)))


def _lib():
    global _loaded
    if _loaded is None:
        lib = _native.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _loaded = lib
    return _loaded


def _code(t):
    import torch
    if t.dtype is torch.bfloat16:
        return LIGER_BF16
    if t.dtype is torch.float32:
        return LIGER_F32
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _same(ref, shape, **named):
    """The tensors that are given are contiguous, on the current device, of ref's dtype and of this shape."""
    for name, t in named.items():
        if t is not None:
            _one(name, t, ref.dtype, shape)


def _one(name, t, dtype, shape):
    import torch
    if not t.is_cuda or not t.is_contiguous() or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on the current device")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")


def _bytes(ws):
    """Pointer and size of a workspace tensor (or None)."""
    if ws is None:
        return None, 0
    _one("ws", ws, ws.dtype, None)
    return ws.data_ptr(), ws.numel() * ws.element_size()


# -------------------------------------------------------------- block norms
def _norm_shapes(z, gate):
    shape = tuple(z.shape)
    cols = shape[-1]
    rows = z.numel() // cols if cols else 0
    gates = 0 if gate is None else gate.numel() // cols if cols else 0
    return shape, rows, cols, gates


def _gate(gate, ref, cols, gates):
    if gate is not None:
        _one("gate", gate, ref.dtype, None)
        if gates < 1 or gate.shape[-1] != cols or gate.dim() > 2:
            raise ValueError(f"gate must be [cols] or [gates, cols] with cols = {cols}, not {tuple(gate.shape)}")


def liger_block_norm_fwd(z, r, h, y=None, w_post=None, gate=None, w_pre=None, rstd_z=None, rstd_h=None,
                         res_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6):
    """h = res_scale r + block_scale gate rmsnorm(z) w_post, y = rmsnorm(h) w_pre (see liger_train.h).

    z, r, h, y [..., cols]; w_post, w_pre [cols] or None; gate None, [cols] or [gates, cols] (gate row i for the i-th
    run of rows / gates rows); rstd_z, rstd_h float32, one per row, or None.  h may be r, and y may be z."""
    shape, rows, cols, gates = _norm_shapes(z, gate)
    _same(z, shape, z=z, r=r, h=h, y=y)
    _same(z, (cols,), w_post=w_post, w_pre=w_pre)
    _gate(gate, z, cols, gates)
    _rows(rows, rstd_z=rstd_z, rstd_h=rstd_h)
    _check(_lib().liger_block_norm_fwd(_ptr(z), _ptr(r), _ptr(w_post), _ptr(gate), _ptr(w_pre), _ptr(h), _ptr(y),
                                       _ptr(rstd_z), _ptr(rstd_h), rows, cols, gates, res_scale, block_scale, eps,
                                       _code(z), _stream()))
    return h, y


def _rows(rows, **named):
    import torch
    for name, t in named.items():
        if t is not None:
            _one(name, t, torch.float32, None)
            if t.numel() != rows:
                raise ValueError(f"{name} must hold {rows} values, not {t.numel()}")


def liger_block_norm_bwd_workspace(rows: int, cols: int, gates: int = 0) -> int:
    return int(_lib().liger_block_norm_bwd_workspace(rows, cols, gates))


def liger_block_norm_bwd(dh, dy, z, h, dr, dz, ws, w_post=None, gate=None, w_pre=None, rstd_z=None, rstd_h=None,
                         dw_post=None, dgate=None, dw_pre=None, res_scale: float = 1.0, block_scale: float = 1.0):
    """Backward of liger_block_norm_fwd (see liger_train.h): dh or None, and dy, give dr, dz and the gradients of the
    weights and of the gate that the forward had.  dr may be dh, and dz may be dy."""
    shape, rows, cols, gates = _norm_shapes(dr, gate)
    _same(dr, shape, dh=dh, dy=dy, z=z, h=h, dr=dr, dz=dz)
    _same(dr, (cols,), w_post=w_post, w_pre=w_pre, dw_post=dw_post, dw_pre=dw_pre)
    _gate(gate, dr, cols, gates)
    if dgate is not None:
        _one("dgate", dgate, dr.dtype, None if gate is None else tuple(gate.shape))
    _rows(rows, rstd_z=rstd_z, rstd_h=rstd_h)
    pws, nws = _bytes(ws)
    _check(_lib().liger_block_norm_bwd(_ptr(dh), _ptr(dy), _ptr(z), _ptr(h), _ptr(w_post), _ptr(gate), _ptr(w_pre),
                                       _ptr(rstd_z), _ptr(rstd_h), _ptr(dr), _ptr(dz), _ptr(dw_post), _ptr(dgate),
                                       _ptr(dw_pre), pws, nws, rows, cols, gates, res_scale, block_scale, _code(dr),
                                       _stream()))
    return dr, dz
