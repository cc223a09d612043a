"""Python binding of the layer-norm layer's operators and of scored logits (``include/liger_layer.h``).

As in ``_native``, every function has the name of the C entry point it calls,
takes torch tensors that already live on the GPU, runs on the current stream
and raises ``LigerError`` on a non-zero status.  What the library cannot see
(device, dtype, shape and strides of the tensors) is checked here and raises
``ValueError`` or ``TypeError``.
"""
from __future__ import annotations

import os
import re

from . import _native
from ._native import _D, _F, _I64, _INT, _P, _SZ, LIGER_BF16, LIGER_F32, _check, _ptr

HEADER = os.path.join(os.path.dirname(_native.PKG), "include", "liger_layer.h")

_ROPE = ([_P] * 5 + [_I64] * 10 + [_INT, _D, _INT] + [_D] * 5 + [_INT, _P], _INT)
SIGNATURES = {
    "liger_layernorm_fwd": ([_P] * 6 + [_I64] * 2 + [_F, _INT, _P], _INT),
    "liger_layernorm_bwd_workspace": ([_I64] * 2, _SZ),
    "liger_layernorm_bwd": ([_P] * 10 + [_SZ] + [_I64] * 2 + [_INT, _P], _INT),
    "liger_linear_act_fwd": ([_P] * 6 + [_I64] * 3 + [_INT] * 2 + [_P], _INT),
    "liger_linear_act_bwd_workspace": ([_I64] * 3 + [_INT] * 2, _SZ),
    "liger_linear_act_bwd": ([_P] * 8 + [_SZ] + [_I64] * 3 + [_INT] * 2 + [_P], _INT),
    "liger_rope_scaled_fwd": _ROPE,
    "liger_rope_scaled_bwd": _ROPE,
    "liger_token_logp_fwd": ([_P, _I64, _P] + [_I64] * 3 + [_F] + [_P] * 4 + [_I64, _P, _P, _INT, _P], _INT),
    "liger_token_logp_bwd": ([_P, _I64] + [_P] * 6 + [_I64] * 3 + [_F, _P, _I64, _INT, _P], _INT),
}

TOP_MAX = 32        # LIGER_TOP_MAX
_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_PAIRINGS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}

_loaded = None
torch = None        # imported with the library, on the first call


def header_functions() -> list:
    """Names of the functions include/liger_layer.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(liger_[a-z_0-9]+)\s*\(", text, re.M)))


def _lib():
    global _loaded, torch
    if _loaded is None:
        import torch as t
        lib = _native.load()
        if t.cuda.is_available():
            t.cuda.init()       # the calls ask for the current device without it
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


def _choice(table, value, what):
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"{what} {value!r}: one of {', '.join(table)}") from None


def _raise(dev, dtype, shape, t):
    """Says what is wrong with a tensor that a check below did not let pass."""
    if t.get_device() != dev:
        raise ValueError(f"tensors must be on the current device, cuda:{dev} (got one on {t.device})")
    if t.dtype is not dtype:
        raise TypeError(f"expected a {dtype} tensor, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"tensors must be contiguous (got strides {tuple(t.stride())})")


# The checks are written for calls of a few microseconds: one pass over the attributes, and words only on failure.
def _like(dev, dtype, shape, *ts):
    """Those of the tensors that are given are contiguous, on device dev, of this dtype and shape."""
    for t in ts:
        if t is not None and (t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev):
            _raise(dev, dtype, shape, t)


def _hold(dev, dtype, n, *ts):
    """As _like, for any shape of n elements."""
    for t in ts:
        if t is not None and (t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != dev):
            _raise(dev, dtype, (n,), t)


def _bytes(dev, ws):
    """Pointer and size of a workspace tensor (or None)."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        _raise(dev, ws.dtype, ws.shape, ws)
    return ws.data_ptr(), ws.numel() * ws.element_size()


# -------------------------------------------------------------- layer norm
def _rows(x):
    cols = x.shape[-1]
    return x.numel() // cols if cols else 0, cols


def liger_layernorm_fwd(x, w, b, y, mean=None, rstd=None, eps: float = 1e-5):
    """y = (x - mean) rstd w + b over the last dimension (see liger_layer.h).

    x, y [..., cols]; w, b [cols] or None; mean, rstd float32, one per row, or None.  y may be x."""
    lib = _loaded or _lib()
    dev, dt = torch._C._cuda_getDevice(), x.dtype
    rows, cols = _rows(x)
    _like(dev, dt, x.shape, x, y)
    _like(dev, dt, x.shape[-1:], w, b)
    _hold(dev, torch.float32, rows, mean, rstd)
    _check(lib.liger_layernorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd), rows, cols, eps, _code(dt),
                                   torch._C._cuda_getCurrentRawStream(dev)))
    return y


def liger_layernorm_bwd_workspace(rows: int, cols: int) -> int:
    return int((_loaded or _lib()).liger_layernorm_bwd_workspace(rows, cols))


def liger_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws, dres=None):
    """Backward of liger_layernorm_fwd: dx (plus dres, the gradient past the norm, if given), dw and db (each may be None).
    dx may be dy or dres."""
    lib = _loaded or _lib()
    dev, dt = torch._C._cuda_getDevice(), x.dtype
    rows, cols = _rows(x)
    _like(dev, dt, x.shape, x, dy, dx, dres)
    _like(dev, dt, x.shape[-1:], w, dw, db)
    _hold(dev, torch.float32, rows, mean, rstd)
    pws, nws = _bytes(dev, ws)
    _check(lib.liger_layernorm_bwd(_ptr(dy), _ptr(dres), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw),
                                   _ptr(db), pws, nws, rows, cols, _code(dt), torch._C._cuda_getCurrentRawStream(dev)))
    return dx, dw, db


# ------------------------------------------------- projection with bias, activation and residual
def _kept_type(dt):
    return torch.float16 if dt is torch.bfloat16 else torch.float32


def liger_linear_act_fwd(X, W, Y, bias=None, residual=None, act: str = "none", pre=None):
    """Y = act(X W^T + bias) + residual (see liger_layer.h).

    X [T, H], W [N, H], Y and residual [T, N], bias [N]; act "none", "relu", "gelu", "gelu_tanh" or "silu"; pre [T, N] or
    None: X W^T + bias kept for the backward, float16 for bfloat16 tensors, else float32.  residual may be Y."""
    lib = _loaded or _lib()
    dev, dt = torch._C._cuda_getDevice(), X.dtype
    T, H = X.shape
    N = W.shape[0]
    _like(dev, dt, (T, H), X)
    _like(dev, dt, (N, H), W)
    _like(dev, dt, (T, N), Y, residual)
    _like(dev, dt, (N,), bias)
    _like(dev, _kept_type(dt), (T, N), pre)
    _check(lib.liger_linear_act_fwd(_ptr(X), _ptr(W), _ptr(bias), _ptr(residual), _ptr(Y), _ptr(pre), T, H, N,
                                    _choice(_ACTS, act, "act"), _code(dt), torch._C._cuda_getCurrentRawStream(dev)))
    return Y


def liger_linear_act_bwd_workspace(T: int, H: int, N: int, act: str = "none", dtype: int = LIGER_BF16) -> int:
    return int((_loaded or _lib()).liger_linear_act_bwd_workspace(T, H, N, _choice(_ACTS, act, "act"), dtype))


def liger_linear_act_bwd(dY, X, W, dX, dW, db, ws, pre=None, act: str = "none"):
    """Backward of liger_linear_act_fwd: dX, dW and db (each may be None) from dY and what the forward kept in pre (None with
    act "none"); ws as liger_linear_act_bwd_workspace says.  The gradient of the residual is dY."""
    lib = _loaded or _lib()
    dev, dt = torch._C._cuda_getDevice(), X.dtype
    T, H = X.shape
    N = W.shape[0]
    _like(dev, dt, (T, H), X, dX)
    _like(dev, dt, (N, H), W, dW)
    _like(dev, dt, (T, N), dY)
    _like(dev, dt, (N,), db)
    _like(dev, _kept_type(dt), (T, N), pre)
    pws, nws = _bytes(dev, ws)
    _check(lib.liger_linear_act_bwd(_ptr(dY), _ptr(X), _ptr(W), _ptr(pre), _ptr(dX), _ptr(dW), _ptr(db), pws, nws, T, H, N,
                                    _choice(_ACTS, act, "act"), _code(dt), torch._C._cuda_getCurrentRawStream(dev)))
    return dX, dW, db


# ------------------------------------------------------------- rotary positions, partial and scaled
def _heads(dev, dt, t, B, S, D):
    """Head count and token stride of a [B, S, heads, D] view (or None: 0 heads)."""
    if t is None:
        return 0, 0
    shape, strides = t.shape, t.stride()
    if len(shape) != 4:
        raise ValueError(f"expected [batch, seq, heads, head_dim], got {tuple(shape)}")
    b, s, h, d = shape
    if b != B or s != S or d != D or t.get_device() != dev or t.dtype is not dt:
        if b == B and s == S and d == D:
            _raise(dev, dt, shape, t)
        raise ValueError(f"expected [batch, seq, heads, head_dim] = [{B}, {S}, heads, {D}], got {tuple(shape)}")
    sb, ss, sh, sd = strides
    if B == 0 or S == 0 or h == 0:
        return h, h * D
    if (sd != 1 and D > 1) or (sh != D and h > 1) or (S > 1 and B > 1 and sb != S * ss):
        raise ValueError(f"heads must stand dense and tokens evenly apart (got strides {strides})")
    return h, ss if S > 1 else sb if B > 1 else h * D


def _rope_scaled(fn, q, k, q_out, k_out, rotary_dim, pos, theta, pairing, scaling, factor, low, high, orig_len, attn_factor):
    lib = _loaded or _lib()
    dev = torch._C._cuda_getDevice()
    ref = q if q is not None else k
    if ref is None or ref.dim() != 4:
        raise ValueError("q or k is required, [batch, seq, heads, head_dim]")
    dt = ref.dtype
    B, S, _, D = ref.shape
    Hq, qs = _heads(dev, dt, q, B, S, D)
    Hk, ks = _heads(dev, dt, k, B, S, D)
    Hqo, qos = (Hq, qs) if q_out is q else _heads(dev, dt, q_out, B, S, D)
    Hko, kos = (Hk, ks) if k_out is k else _heads(dev, dt, k_out, B, S, D)
    if Hqo != Hq or Hko != Hk:
        raise ValueError(f"outputs have {Hqo} and {Hko} heads, inputs {Hq} and {Hk}")
    _like(dev, torch.int32, (B, S), pos)
    _check(getattr(lib, fn)(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(pos), B, S, Hq, Hk, D, rotary_dim, qs, ks, qos,
                            kos, _choice(_PAIRINGS, pairing, "pairing"), theta, _choice(_SCALINGS, scaling, "scaling"), factor,
                            low, high, orig_len, attn_factor, _code(dt), torch._C._cuda_getCurrentRawStream(dev)))
    return q_out, k_out


def liger_rope_scaled_fwd(q, k, q_out, k_out, rotary_dim: int, pos=None, theta: float = 1e4, pairing: str = "half",
                          scaling: str = "none", factor: float = 1.0, low: float = 1.0, high: float = 32.0,
                          orig_len: float = 0.0, attn_factor: float = 0.0):
    """Rotates the first rotary_dim elements of each head of q and k by the token's position, the rest copied (see
    liger_layer.h for the frequencies of scaling "none", "linear", "ntk", "bands" and "yarn").

    q, k, q_out, k_out [batch, seq, heads, head_dim]: views with dense heads and evenly spaced tokens (a slice of a packed
    projection); q_out may be q and k_out k (in place); q with q_out, or k with k_out, may be None.  pos int32 [batch, seq]
    or None (0, 1, ...).  pairing "half" (i, i + rotary_dim / 2) or "interleaved" (2i, 2i + 1)."""
    return _rope_scaled("liger_rope_scaled_fwd", q, k, q_out, k_out, rotary_dim, pos, theta, pairing, scaling, factor, low,
                        high, orig_len, attn_factor)


def liger_rope_scaled_bwd(dq, dk, dq_out, dk_out, rotary_dim: int, pos=None, theta: float = 1e4, pairing: str = "half",
                          scaling: str = "none", factor: float = 1.0, low: float = 1.0, high: float = 32.0,
                          orig_len: float = 0.0, attn_factor: float = 0.0):
    """The transpose of liger_rope_scaled_fwd: from the gradients of its outputs to those of q and k."""
    return _rope_scaled("liger_rope_scaled_bwd", dq, dk, dq_out, dk_out, rotary_dim, pos, theta, pairing, scaling, factor, low,
                        high, orig_len, attn_factor)


# ------------------------------------------------ token log-probabilities, entropy, alternatives
def _logit_rows(dev, t, T, V, dt):
    """Row stride of [T, V] logits (dense rows)."""
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] != V or t.get_device() != dev or t.dtype is not dt or \
            (V > 1 and t.stride(1) != 1):
        _raise(dev, dt, (T, V), t)
    return t.stride(0) if T > 1 else V


def liger_token_logp_fwd(logits, tokens, logp, row_max=None, log_sum=None, entropy=None, top_logp=None, top_ids=None,
                         temperature: float = 1.0, ignore_index: int = -100):
    """Of the distributions softmax(logits / temperature): the log-probability of each row's token (0 at ignore_index), the
    row's largest logit and log sum exp((logits - row_max) / temperature), the entropy, and the top_ids.shape[1] (at most
    32) likeliest tokens with their log-probabilities (see liger_layer.h).

    logits [T, V] with dense rows (any row stride); tokens int64 [T] with logp float32 [T], or both None; row_max, log_sum,
    entropy float32 [T] or None; top_logp float32 with top_ids int64 [T, k], or both None."""
    lib = _loaded or _lib()
    dev, f32 = torch._C._cuda_getDevice(), torch.float32
    T, V = logits.shape
    dt = logits.dtype
    ld = _logit_rows(dev, logits, T, V, dt)
    _like(dev, torch.int64, (T,), tokens)
    _hold(dev, f32, T, logp, row_max, log_sum, entropy)
    k = 0
    if top_ids is not None:
        k = top_ids.shape[-1] if top_ids.dim() == 2 else -1
        _like(dev, torch.int64, (T, k), top_ids)
        _like(dev, f32, (T, k), top_logp)
        if k == 0:
            top_ids = top_logp = None
    _check(lib.liger_token_logp_fwd(_ptr(logits), ld, _ptr(tokens), T, V, ignore_index, temperature, _ptr(logp),
                                    _ptr(row_max), _ptr(log_sum), _ptr(entropy), k, _ptr(top_logp), _ptr(top_ids), _code(dt),
                                    torch._C._cuda_getCurrentRawStream(dev)))
    return logp


def liger_token_logp_bwd(logits, tokens, row_max, log_sum, g_logp, dlogits, entropy=None, g_entropy=None,
                         temperature: float = 1.0, ignore_index: int = -100):
    """The gradient of the logits from g_logp and g_entropy (float32 [T], either may be None), with row_max, log_sum and
    entropy as liger_token_logp_fwd wrote them.  dlogits may be logits."""
    lib = _loaded or _lib()
    dev, f32 = torch._C._cuda_getDevice(), torch.float32
    T, V = logits.shape
    dt = logits.dtype
    ld, ldd = _logit_rows(dev, logits, T, V, dt), _logit_rows(dev, dlogits, T, V, dt)
    _like(dev, torch.int64, (T,), tokens)
    _hold(dev, f32, T, row_max, log_sum, entropy, g_logp, g_entropy)
    _check(lib.liger_token_logp_bwd(_ptr(logits), ld, _ptr(tokens), _ptr(row_max), _ptr(log_sum), _ptr(entropy),
                                    _ptr(g_logp), _ptr(g_entropy), T, V, ignore_index, temperature, _ptr(dlogits), ldd,
                                    _code(dt), torch._C._cuda_getCurrentRawStream(dev)))
    return dlogits
