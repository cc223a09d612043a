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
    "liger_swiglu_fwd_ckpt8": ([_P] * 7 + [_I64] * 2 + [_INT, _P], _INT),
    "liger_swiglu_bwd_ckpt8": ([_P] * 7 + [_I64] * 2 + [_INT, _P], _INT),
    "liger_fused_linear_swiglu_fwd_ckpt8": ([_P] * 8 + [_I64] * 3 + [_INT, _P], _INT),
    "liger_fused_linear_swiglu_bwd_ckpt8": ([_P] * 12 + [_SZ] + [_I64] * 3 + [_INT, _P], _INT),
    "liger_linear_logp_workspace": ([_I64] * 3 + [_INT], _SZ),
    "liger_linear_logp_fwd": ([_P] * 3 + [_I64] * 4 + [_P] * 2 + [_SZ, _INT, _P], _INT),
    "liger_linear_logp_fwd_async": ([_P] * 3 + [_I64] * 4 + [_P] * 2 + [_SZ, _INT, _P], _INT),
    "liger_linear_policy_workspace": ([_I64] * 5 + [_INT], _SZ),
    "liger_linear_policy_fwd_bwd": ([_P] * 7 + [_I64] * 5 + [_INT] * 2 + [_F] * 4 + [_P] * 6 + [_SZ, _I64, _INT, _P], _INT),
    "liger_linear_policy_fwd_bwd_async": ([_P] * 7 + [_I64] * 5 + [_INT] * 2 + [_F] * 4 + [_P] * 6
                                          + [_SZ, _I64, _INT, _P], _INT),
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


# ------------------------------------------------- SwiGLU with 8-bit checkpoints
CKPT8_GROUP = 32    # columns of a row that share a scale byte


def liger_ckpt8_empty(rows: int, cols: int, device="cuda"):
    """An empty 8-bit checkpoint of a [rows, cols] tensor: int8 codes [rows, cols] and uint8 scales
    [rows, ceil(cols / 32)]."""
    import torch
    return (torch.empty(rows, cols, dtype=torch.int8, device=device),
            torch.empty(rows, -(-cols // CKPT8_GROUP), dtype=torch.uint8, device=device))


def _ckpt(rows, cols, *pairs):
    import torch
    groups = -(-cols // CKPT8_GROUP)
    for name, codes, scale in pairs:
        _one(name + "8", codes, torch.int8, None)
        _one(name + "_scale", scale, torch.uint8, None)
        if codes.numel() != rows * cols or scale.numel() != rows * groups:
            raise ValueError(f"the checkpoint of {name} must hold {rows} x {cols} codes and {rows} x {groups} scales")


def liger_swiglu_fwd_ckpt8(gate, up, y, gate8, gate_scale, up8, up_scale):
    """y = silu(gate) up, and the 8-bit checkpoints of gate and up (see liger_train.h); gate, up, y [..., cols]."""
    shape, cols = tuple(gate.shape), gate.shape[-1]
    rows = gate.numel() // cols if cols else 0
    _same(gate, shape, gate=gate, up=up, y=y)
    _ckpt(rows, cols, ("gate", gate8, gate_scale), ("up", up8, up_scale))
    _check(_lib().liger_swiglu_fwd_ckpt8(_ptr(gate), _ptr(up), _ptr(y), _ptr(gate8), _ptr(gate_scale), _ptr(up8),
                                         _ptr(up_scale), rows, cols, _code(gate), _stream()))
    return y


def liger_swiglu_bwd_ckpt8(dy, gate8, gate_scale, up8, up_scale, dgate, dup):
    """dgate and dup from dy and the checkpoints that liger_swiglu_fwd_ckpt8 wrote."""
    shape, cols = tuple(dy.shape), dy.shape[-1]
    rows = dy.numel() // cols if cols else 0
    _same(dy, shape, dy=dy, dgate=dgate, dup=dup)
    _ckpt(rows, cols, ("gate", gate8, gate_scale), ("up", up8, up_scale))
    _check(_lib().liger_swiglu_bwd_ckpt8(_ptr(dy), _ptr(gate8), _ptr(gate_scale), _ptr(up8), _ptr(up_scale), _ptr(dgate),
                                         _ptr(dup), rows, cols, _code(dy), _stream()))
    return dgate, dup


def liger_fused_linear_swiglu_fwd_ckpt8(X, Wg, Wu, out, gate8, gate_scale, up8, up_scale):
    """FusedLinearSwiGLU forward that keeps X Wg^T and X Wu^T in 8 bits."""
    T, H = X.shape
    I = Wg.shape[0]
    _same(X, (T, H), X=X)
    _same(X, (I, H), Wg=Wg, Wu=Wu)
    _same(X, (T, I), out=out)
    _ckpt(T, I, ("gate", gate8, gate_scale), ("up", up8, up_scale))
    _check(_lib().liger_fused_linear_swiglu_fwd_ckpt8(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(out), _ptr(gate8),
                                                      _ptr(gate_scale), _ptr(up8), _ptr(up_scale), T, H, I, _code(X),
                                                      _stream()))
    return out


def liger_fused_linear_swiglu_bwd_ckpt8(X, Wg, Wu, dH, gate8, gate_scale, up8, up_scale, dX, dWg, dWu, ws):
    """FusedLinearSwiGLU backward from the 8-bit checkpoints; ws as liger_fused_linear_swiglu_workspace says."""
    T, H = X.shape
    I = Wg.shape[0]
    _same(X, (T, H), X=X, dX=dX)
    _same(X, (I, H), Wg=Wg, Wu=Wu, dWg=dWg, dWu=dWu)
    _same(X, (T, I), dH=dH)
    _ckpt(T, I, ("gate", gate8, gate_scale), ("up", up8, up_scale))
    pws, nws = _bytes(ws)
    _check(_lib().liger_fused_linear_swiglu_bwd_ckpt8(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(dH), _ptr(gate8),
                                                      _ptr(gate_scale), _ptr(up8), _ptr(up_scale), _ptr(dX), _ptr(dWg),
                                                      _ptr(dWu), pws, nws, T, H, I, _code(X), _stream()))
    return dX, dWg, dWu


# ------------------------------------------------------- heads: label log-probabilities, policy loss
def _head(X, W, labels):
    import torch
    T, H = X.shape
    V = W.shape[0]
    _same(X, (T, H), X=X)
    _same(X, (V, H), W=W)
    _one("labels", labels, torch.int64, (T,))
    return T, H, V


def liger_linear_logp_workspace(T: int, H: int, V: int, dtype: int = LIGER_BF16) -> int:
    return int(_lib().liger_linear_logp_workspace(T, H, V, dtype))


def liger_linear_logp_fwd(X, W, labels, logp, ws, ignore_index: int = -100, wait: bool = True):
    """logp[t] = log softmax(W x_t)[labels[t]], 0 where the label is ignore_index (see liger_train.h); wait=False calls
    the _async form (no host wait: capturable in a CUDA graph; a bad label's logp is NaN)."""
    T, H, V = _head(X, W, labels)
    _rows(T, logp=logp)
    pws, nws = _bytes(ws)
    fn = _lib().liger_linear_logp_fwd if wait else _lib().liger_linear_logp_fwd_async
    _check(fn(_ptr(X), _ptr(W), _ptr(labels), T, H, V, int(ignore_index), _ptr(logp), pws, nws, _code(X), _stream()))
    return logp


_REDUCTION = {"token_mean": 0, "sum": 1, "seq_mean": 2}


def liger_linear_policy_workspace(T: int, H: int, V: int, B: int = 1, chunk: int = 0, dtype: int = LIGER_BF16) -> int:
    return int(_lib().liger_linear_policy_workspace(T, H, V, B, chunk, dtype))


def liger_linear_policy_fwd_bwd(X, W, labels, old_logp, adv, loss, dX, dW, ws, ref_logp=None, cu_seqlens=None, logp=None,
                                stats=None, ignore_index: int = -100, reduction: str = "token_mean", eps_low: float = 0.2,
                                eps_high: float = 0.2, beta: float = 0.0, grad_scale: float = 1.0,
                                adv_per_token: bool = False, chunk: int = 0, wait: bool = True):
    """Clipped policy loss with a KL term, and its gradients dX and dW (each may be None), from the hidden states X [T, H]
    and the head W [V, H] (see liger_train.h).

    labels int64 [T]; old_logp, ref_logp float32 [T]; adv float32, one per sequence ([B]) or, with adv_per_token, one per
    token ([T]); cu_seqlens int32 [B + 1] or None (one sequence); reduction "token_mean", "seq_mean" or "sum"; stats
    float32 [2] or None (mean KL, share of clipped tokens).  wait=False calls the _async form."""
    import torch
    T, H, V = _head(X, W, labels)
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None:
        _one("cu_seqlens", cu_seqlens, torch.int32, (B + 1,))
    _rows(T, old_logp=old_logp, ref_logp=ref_logp, logp=logp)
    _rows(T if adv_per_token else B, adv=adv)
    _rows(1, loss=loss)
    _rows(2, stats=stats)
    _same(X, (T, H), dX=dX)
    _same(X, (V, H), dW=dW)
    pws, nws = _bytes(ws)
    fn = _lib().liger_linear_policy_fwd_bwd if wait else _lib().liger_linear_policy_fwd_bwd_async
    _check(fn(_ptr(X), _ptr(W), _ptr(labels), _ptr(cu_seqlens), _ptr(old_logp), _ptr(ref_logp), _ptr(adv), T, H, V, B,
              int(ignore_index), _REDUCTION[reduction], 1 if adv_per_token else 0, eps_low, eps_high, beta, grad_scale,
              _ptr(loss), _ptr(stats), _ptr(logp), _ptr(dX), _ptr(dW), pws, nws, int(chunk), _code(X), _stream()))
    return loss, dX, dW
