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
from ._native import _F, _I64, _INT, _P, _SZ, LIGER_BF16, LIGER_F32, _check, _ptr

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
torch = None        # imported with the library, on the first call


def header_functions() -> list:
    """Names of the functions include/liger_train.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(liger_[a-z_0-9]+)\s*\(", text, re.M)))


def _lib():
    global _loaded, torch
    if _loaded is None:
        import torch as t
        lib = _native.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        torch = t
        _loaded = lib
    return _loaded


def _code(dtype):
    if dtype is torch.bfloat16:
        return LIGER_BF16
    if dtype is torch.float32:
        return LIGER_F32
    raise TypeError(f"unsupported dtype {dtype}: float32 or bfloat16")


def _raise(dev, dtype, shape, t):
    """Says what is wrong with a tensor that a check below did not let pass."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"tensors must be contiguous CUDA tensors on the current device (got one on {t.device}, "
                         f"strides {tuple(t.stride())})")
    if t.dtype is not dtype:
        raise TypeError(f"expected a {dtype} tensor, got {t.dtype}")
    raise ValueError(f"expected shape {tuple(shape)}, got {tuple(t.shape)}")


# The checks are written for calls of a few microseconds: one pass over the attributes, and words only on failure.
def _like(dev, dtype, shape, *ts):
    """Those of the tensors that are given are contiguous, on device dev, of this dtype and shape."""
    for t in ts:
        if t is not None and (t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()):
            _raise(dev, dtype, shape, t)


def _hold(dev, dtype, n, *ts):
    """As _like, for any shape of n elements."""
    for t in ts:
        if t is not None and (t.get_device() != dev or t.dtype is not dtype or t.numel() != n or not t.is_contiguous()):
            _raise(dev, dtype, (n,), t)


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _bytes(dev, ws):
    """Pointer and size of a workspace tensor (or None)."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        _raise(dev, ws.dtype, ws.shape, ws)
    return ws.data_ptr(), ws.numel() * ws.element_size()


# -------------------------------------------------------------- block norms
def _norm_sizes(dev, ref, gate, w_post, w_pre):
    """shape, rows, cols, gates of the rows `ref` and its checked weights and gate."""
    shape = ref.shape
    cols = shape[-1]
    rows = ref.numel() // cols if cols else 0
    _like(dev, ref.dtype, shape[-1:], w_post, w_pre)
    gates = 0
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != cols or gate.numel() == 0:
            raise ValueError(f"gate must be [cols] or [gates, cols] with cols = {cols}, not {tuple(gate.shape)}")
        _like(dev, ref.dtype, gate.shape, gate)
        gates = gate.numel() // cols
    return shape, rows, cols, gates


def liger_block_norm_fwd(z, r, h, y=None, w_post=None, gate=None, w_pre=None, rstd_z=None, rstd_h=None,
                         res_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6):
    """h = res_scale r + block_scale gate rmsnorm(z) w_post, y = rmsnorm(h) w_pre (see liger_train.h).

    z, r, h, y [..., cols]; w_post, w_pre [cols] or None; gate None, [cols] or [gates, cols] (gate row i for the i-th
    run of rows / gates rows); rstd_z, rstd_h float32, one per row, or None.  h may be r, and y may be z."""
    lib = _loaded or _lib()
    dev, dt = torch.cuda.current_device(), z.dtype
    shape, rows, cols, gates = _norm_sizes(dev, z, gate, w_post, w_pre)
    _like(dev, dt, shape, z, r, h, y)
    _hold(dev, torch.float32, rows, rstd_z, rstd_h)
    _check(lib.liger_block_norm_fwd(_ptr(z), _ptr(r), _ptr(w_post), _ptr(gate), _ptr(w_pre), _ptr(h), _ptr(y),
                                    _ptr(rstd_z), _ptr(rstd_h), rows, cols, gates, res_scale, block_scale, eps, _code(dt),
                                    _raw_stream(dev)))
    return h, y


def liger_block_norm_bwd_workspace(rows: int, cols: int, gates: int = 0) -> int:
    return int(_lib().liger_block_norm_bwd_workspace(rows, cols, gates))


def liger_block_norm_bwd(dh, dy, z, h, dr, dz, ws, w_post=None, gate=None, w_pre=None, rstd_z=None, rstd_h=None,
                         dw_post=None, dgate=None, dw_pre=None, res_scale: float = 1.0, block_scale: float = 1.0):
    """Backward of liger_block_norm_fwd (see liger_train.h): dh or None, and dy, give dr, dz and the gradients of the
    weights and of the gate that the forward had.  dr may be dh, and dz may be dy."""
    lib = _loaded or _lib()
    dev, dt = torch.cuda.current_device(), dr.dtype
    shape, rows, cols, gates = _norm_sizes(dev, dr, gate, w_post, w_pre)
    _like(dev, dt, shape, dh, dy, z, h, dr, dz)
    _like(dev, dt, shape[-1:], dw_post, dw_pre)
    if gate is not None:
        _like(dev, dt, gate.shape, dgate)
    _hold(dev, torch.float32, rows, rstd_z, rstd_h)
    pws, nws = _bytes(dev, ws)
    _check(lib.liger_block_norm_bwd(_ptr(dh), _ptr(dy), _ptr(z), _ptr(h), _ptr(w_post), _ptr(gate), _ptr(w_pre),
                                    _ptr(rstd_z), _ptr(rstd_h), _ptr(dr), _ptr(dz), _ptr(dw_post), _ptr(dgate),
                                    _ptr(dw_pre), pws, nws, rows, cols, gates, res_scale, block_scale, _code(dt),
                                    _raw_stream(dev)))
    return dr, dz


# ------------------------------------------------- SwiGLU with 8-bit checkpoints
CKPT8_GROUP = 32    # columns of a row that share a scale byte


def liger_ckpt8_empty(rows: int, cols: int, device="cuda"):
    """An empty 8-bit checkpoint of a [rows, cols] tensor: int8 codes [rows, cols] and uint8 scales
    [rows, ceil(cols / 32)]."""
    _lib()
    return (torch.empty(rows, cols, dtype=torch.int8, device=device),
            torch.empty(rows, -(-cols // CKPT8_GROUP), dtype=torch.uint8, device=device))


def _ckpt(dev, rows, cols, gate8, gate_scale, up8, up_scale):
    _hold(dev, torch.int8, rows * cols, gate8, up8)
    _hold(dev, torch.uint8, rows * -(-cols // CKPT8_GROUP), gate_scale, up_scale)


def liger_swiglu_fwd_ckpt8(gate, up, y, gate8, gate_scale, up8, up_scale):
    """y = silu(gate) up, and the 8-bit checkpoints of gate and up (see liger_train.h); gate, up, y [..., cols]."""
    lib = _loaded or _lib()
    dev, dt, shape = torch.cuda.current_device(), gate.dtype, gate.shape
    cols = shape[-1]
    rows = gate.numel() // cols if cols else 0
    _like(dev, dt, shape, gate, up, y)
    _ckpt(dev, rows, cols, gate8, gate_scale, up8, up_scale)
    _check(lib.liger_swiglu_fwd_ckpt8(_ptr(gate), _ptr(up), _ptr(y), _ptr(gate8), _ptr(gate_scale), _ptr(up8),
                                      _ptr(up_scale), rows, cols, _code(dt), _raw_stream(dev)))
    return y


def liger_swiglu_bwd_ckpt8(dy, gate8, gate_scale, up8, up_scale, dgate, dup):
    """dgate and dup from dy and the checkpoints that liger_swiglu_fwd_ckpt8 wrote."""
    lib = _loaded or _lib()
    dev, dt, shape = torch.cuda.current_device(), dy.dtype, dy.shape
    cols = shape[-1]
    rows = dy.numel() // cols if cols else 0
    _like(dev, dt, shape, dy, dgate, dup)
    _ckpt(dev, rows, cols, gate8, gate_scale, up8, up_scale)
    _check(lib.liger_swiglu_bwd_ckpt8(_ptr(dy), _ptr(gate8), _ptr(gate_scale), _ptr(up8), _ptr(up_scale), _ptr(dgate),
                                      _ptr(dup), rows, cols, _code(dt), _raw_stream(dev)))
    return dgate, dup


def liger_fused_linear_swiglu_fwd_ckpt8(X, Wg, Wu, out, gate8, gate_scale, up8, up_scale):
    """FusedLinearSwiGLU forward that keeps X Wg^T and X Wu^T in 8 bits."""
    lib = _loaded or _lib()
    dev, dt = torch.cuda.current_device(), X.dtype
    T, H = X.shape
    I = Wg.shape[0]
    _like(dev, dt, (T, H), X)
    _like(dev, dt, (I, H), Wg, Wu)
    _like(dev, dt, (T, I), out)
    _ckpt(dev, T, I, gate8, gate_scale, up8, up_scale)
    _check(lib.liger_fused_linear_swiglu_fwd_ckpt8(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(out), _ptr(gate8), _ptr(gate_scale),
                                                   _ptr(up8), _ptr(up_scale), T, H, I, _code(dt), _raw_stream(dev)))
    return out


def liger_fused_linear_swiglu_bwd_ckpt8(X, Wg, Wu, dH, gate8, gate_scale, up8, up_scale, dX, dWg, dWu, ws):
    """FusedLinearSwiGLU backward from the 8-bit checkpoints; ws as liger_fused_linear_swiglu_workspace says."""
    lib = _loaded or _lib()
    dev, dt = torch.cuda.current_device(), X.dtype
    T, H = X.shape
    I = Wg.shape[0]
    _like(dev, dt, (T, H), X, dX)
    _like(dev, dt, (I, H), Wg, Wu, dWg, dWu)
    _like(dev, dt, (T, I), dH)
    _ckpt(dev, T, I, gate8, gate_scale, up8, up_scale)
    pws, nws = _bytes(dev, ws)
    _check(lib.liger_fused_linear_swiglu_bwd_ckpt8(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(dH), _ptr(gate8), _ptr(gate_scale),
                                                   _ptr(up8), _ptr(up_scale), _ptr(dX), _ptr(dWg), _ptr(dWu), pws, nws, T,
                                                   H, I, _code(dt), _raw_stream(dev)))
    return dX, dWg, dWu


# ------------------------------------------------------- heads: label log-probabilities, policy loss
def _head(dev, X, W, labels):
    T, H = X.shape
    V = W.shape[0]
    _like(dev, X.dtype, (T, H), X)
    _like(dev, X.dtype, (V, H), W)
    _like(dev, torch.int64, (T,), labels)
    return T, H, V


def liger_linear_logp_workspace(T: int, H: int, V: int, dtype: int = LIGER_BF16) -> int:
    return int(_lib().liger_linear_logp_workspace(T, H, V, dtype))


def liger_linear_logp_fwd(X, W, labels, logp, ws, ignore_index: int = -100, wait: bool = True):
    """logp[t] = log softmax(W x_t)[labels[t]], 0 where the label is ignore_index (see liger_train.h); wait=False calls
    the _async form (no host wait: capturable in a CUDA graph; a bad label's logp is NaN)."""
    lib = _loaded or _lib()
    dev = torch.cuda.current_device()
    T, H, V = _head(dev, X, W, labels)
    _hold(dev, torch.float32, T, logp)
    pws, nws = _bytes(dev, ws)
    fn = lib.liger_linear_logp_fwd if wait else lib.liger_linear_logp_fwd_async
    _check(fn(_ptr(X), _ptr(W), _ptr(labels), T, H, V, ignore_index, _ptr(logp), pws, nws, _code(X.dtype),
              _raw_stream(dev)))
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
    float32 [2] or None (mean KL, share of clipped tokens); logp float32 [T] or None, no tensor of the inputs.  wait=False calls
    the _async form."""
    lib = _loaded or _lib()
    dev, f32 = torch.cuda.current_device(), torch.float32
    T, H, V = _head(dev, X, W, labels)
    B = 1
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        _like(dev, torch.int32, (B + 1,), cu_seqlens)
    _hold(dev, f32, T, old_logp, ref_logp, logp)
    _hold(dev, f32, T if adv_per_token else B, adv)
    _hold(dev, f32, 1, loss)
    _hold(dev, f32, 2, stats)
    _like(dev, X.dtype, (T, H), dX)
    _like(dev, X.dtype, (V, H), dW)
    pws, nws = _bytes(dev, ws)
    fn = lib.liger_linear_policy_fwd_bwd if wait else lib.liger_linear_policy_fwd_bwd_async
    _check(fn(_ptr(X), _ptr(W), _ptr(labels), _ptr(cu_seqlens), _ptr(old_logp), _ptr(ref_logp), _ptr(adv), T, H, V, B,
              ignore_index, _REDUCTION[reduction], 1 if adv_per_token else 0, eps_low, eps_high, beta, grad_scale,
              _ptr(loss), _ptr(stats), _ptr(logp), _ptr(dX), _ptr(dW), pws, nws, chunk, _code(X.dtype),
              _raw_stream(dev)))
    return loss, dX, dW
