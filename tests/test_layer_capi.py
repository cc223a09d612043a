"""The C entry points of include/liger_layer.h: all exported and bound, and their argument checks (host only: no CUDA call)."""
import ctypes
import os

import pytest

from transformer_rmsnorm_fwd_gb300 import _layer, _native

OK, ODD, ODDER = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1001)   # never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        from transformer_rmsnorm_fwd_gb300 import build
        build.build()
    return _layer._lib()


def test_exports_every_declared_function(lib):
    names = _layer.header_functions()
    assert names and set(names) == set(_layer.SIGNATURES)
    import transformer_rmsnorm_fwd_gb300 as L
    for n in names:
        assert hasattr(lib, n) and hasattr(L, n), n
    with open(_layer.HEADER) as f:
        text = f.read()
    assert f"#define LIGER_TOP_MAX {_layer.TOP_MAX}\n" in text
    for table, prefix in ((_layer._ACTS, "LIGER_ACT_"), (_layer._SCALINGS, "LIGER_ROPE_")):
        for name, code in table.items():
            assert f"#define {prefix}{name.upper()} {code}\n" in text


def _call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*a.values(), None)


def test_layernorm_checks(lib):
    base = dict(x=OK, w=OK, b=OK, y=OK, mean=OK, rstd=OK, rows=5, cols=64, eps=1e-5, dtype=1)
    fwd = lambda **kw: _call(lib.liger_layernorm_fwd, base, kw)     # noqa: E731
    assert fwd(dtype=2) == -3 and fwd(rows=-1) == -2 and fwd(cols=0) == -2 and fwd(cols=(1 << 24) + 1) == -2
    assert fwd(rows=1 << 46, cols=1 << 20) == -2
    assert fwd(eps=-1.0) == -2 and fwd(eps=NAN) == -2
    assert fwd(x=None) == -1 and fwd(y=None) == -1
    for k in ("x", "w", "b", "y"):
        assert fwd(**{k: ODD}) == -4
    assert fwd(mean=ODDER) == -4 and fwd(rstd=ODDER) == -4
    assert fwd(rows=0, x=None, y=None) == 0
    need = lib.liger_layernorm_bwd_workspace(5, 64)
    assert need == 2 * 5 * 64 * 4 and lib.liger_layernorm_bwd_workspace(1 << 20, 8) == 2 * 1024 * 8 * 4
    assert lib.liger_layernorm_bwd_workspace(0, 64) == 0 and lib.liger_layernorm_bwd_workspace(5, -1) == 0
    base = dict(dy=OK, dres=OK, x=OK, w=OK, mean=OK, rstd=OK, dx=OK, dw=OK, db=OK, ws=OK, ws_bytes=need, rows=5, cols=64, dtype=0)
    bwd = lambda **kw: _call(lib.liger_layernorm_bwd, base, kw)     # noqa: E731
    assert bwd(dtype=-1) == -3 and bwd(cols=0) == -2 and bwd(rows=-3) == -2
    for k in ("dy", "x", "mean", "rstd", "dx"):
        assert bwd(**{k: None}) == -1
    for k in ("dy", "dres", "x", "w", "dx", "dw", "db"):
        assert bwd(**{k: ODD}) == -4
    assert bwd(ws=None) == -6 and bwd(ws_bytes=need - 1) == -6 and bwd(ws=ODD) == -6
    assert "workspace" in lib.liger_last_error().decode()
    assert bwd(rows=0, dw=None, db=None, x=None) == 0


def test_linear_act_checks(lib):
    base = dict(X=OK, W=OK, bias=OK, residual=OK, Y=OK, pre=OK, T=5, H=64, N=72, act=1, dtype=1)
    fwd = lambda **kw: _call(lib.liger_linear_act_fwd, base, kw)    # noqa: E731
    assert fwd(dtype=3) == -3
    for kw in (dict(T=-1), dict(H=0), dict(N=0), dict(N=-5), dict(act=5), dict(act=-1), dict(H=1 << 31), dict(T=1 << 29, N=1 << 29)):
        assert fwd(**kw) == -2, kw
    for k in ("X", "W", "Y"):
        assert fwd(**{k: None}) == -1
    for k in ("X", "W", "bias", "residual", "Y", "pre"):
        assert fwd(**{k: ODD}) == -4
    assert fwd(T=0, X=None) == 0
    size = lib.liger_linear_act_bwd_workspace
    assert size(0, 64, 64, 1, 1) == 0 and size(5, 64, 64, 9, 1) == 0 and size(5, 64, 64, 1, 4) == 0 and size(5, -1, 64, 1, 1) == 0
    assert lib.liger_last_error() == b""
    assert size(100, 64, 72, 0, 1) < size(100, 64, 72, 2, 1) <= size(100, 64, 72, 2, 0)
    need = size(5, 64, 72, 1, 1)
    base = dict(dY=OK, X=OK, W=OK, pre=OK, dX=OK, dW=OK, db=OK, ws=OK, ws_bytes=need, T=5, H=64, N=72, act=1, dtype=1)
    bwd = lambda **kw: _call(lib.liger_linear_act_bwd, base, kw)    # noqa: E731
    assert bwd(dtype=7) == -3 and bwd(act=6) == -2 and bwd(H=0) == -2
    for k in ("dY", "X", "W", "pre"):
        assert bwd(**{k: None}) == -1
    for k in ("dY", "X", "W", "pre", "dX", "dW", "db"):
        assert bwd(**{k: ODD}) == -4
    assert bwd(ws=None) == -6 and bwd(ws_bytes=need - 1) == -6 and bwd(ws=ctypes.c_void_p(0x1010)) == -6


def _rope_args(kw):
    return dict(dict(q=OK, k=OK, qo=ctypes.c_void_p(0x9000), ko=ctypes.c_void_p(0xA000), pos=None, B=2, S=3, Hq=4, Hk=2, D=64,
                     R=32, qs=256, ks=128, qos=256, kos=128, pairing=0, theta=1e4, scaling=4, factor=4.0, low=1.0, high=32.0,
                     orig=4096.0, attn=0.0, dtype=1), **kw)


@pytest.mark.parametrize("name", ["liger_rope_scaled_fwd", "liger_rope_scaled_bwd"])
def test_rope_scaled_checks(lib, name):
    run = lambda **kw: getattr(lib, name)(*_rope_args(kw).values(), None)   # noqa: E731
    assert run(dtype=2) == -3
    for kw in (dict(B=-1), dict(S=-1), dict(Hq=-1), dict(D=0), dict(D=513, qs=4096, qos=4096), dict(R=0), dict(R=31), dict(R=66),
               dict(pairing=2), dict(qs=255), dict(kos=127), dict(theta=0.0), dict(theta=INF), dict(scaling=5), dict(scaling=-1),
               dict(factor=0.0), dict(factor=NAN), dict(orig=0.0), dict(low=0.0), dict(high=-1.0), dict(theta=1.0),
               dict(scaling=3, low=4.0, high=4.0), dict(scaling=3, low=NAN), dict(attn=INF), dict(B=1 << 30, S=1 << 30),
               dict(qs=1 << 60, qos=1 << 60, S=1 << 20), dict(scaling=2, factor=1e300, R=4)):
        assert run(**kw) == -2, kw
    for k in ("q", "k", "qo", "ko"):
        assert run(**{k: None}) == -1
        assert run(**{k: ODDER}) == -4
    assert run(pos=ODDER) == -4
    assert run(qo=OK, q=OK, qos=512) == -2          # in place with another stride
    assert run(B=0, q=None) == 0 and run(Hq=0, Hk=0, q=None, k=None, qo=None, ko=None) == 0


def test_token_logp_checks(lib):
    base = dict(z=OK, ld=100, tokens=OK, T=5, V=100, ignore=-100, temp=1.0, logp=OK, row_max=OK, log_sum=OK, entropy=OK, k=4,
                top_logp=OK, top_ids=OK, dtype=1)
    fwd = lambda **kw: _call(lib.liger_token_logp_fwd, base, kw)    # noqa: E731
    assert fwd(dtype=2) == -3
    for kw in (dict(T=-1), dict(V=0), dict(ld=99), dict(temp=0.0), dict(temp=-1.0), dict(temp=NAN), dict(temp=INF), dict(temp=1e-40),
               dict(k=-1), dict(k=33), dict(V=3, ld=100, k=4), dict(T=1 << 31), dict(V=1 << 31, ld=1 << 32)):
        assert fwd(**kw) == -2, kw
    assert fwd(z=None) == -1 and fwd(tokens=None) == -1 and fwd(logp=None) == -1 and fwd(top_ids=None) == -1
    assert fwd(k=0) == -1 and fwd(top_logp=None) == -1
    for k in ("z", "tokens", "logp", "row_max", "log_sum", "entropy", "top_logp", "top_ids"):
        assert fwd(**{k: ODDER}) == -4
    assert fwd(T=0, z=None) == 0
    base = dict(z=OK, ld=100, tokens=OK, row_max=OK, log_sum=OK, entropy=OK, g_logp=OK, g_entropy=OK, T=5, V=100, ignore=-100,
                temp=1.0, dz=ctypes.c_void_p(0x9000), ldd=100, dtype=0)
    bwd = lambda **kw: _call(lib.liger_token_logp_bwd, base, kw)    # noqa: E731
    assert bwd(dtype=2) == -3 and bwd(ldd=99) == -2 and bwd(temp=0.0) == -2 and bwd(dz=OK, ldd=128) == -2
    for k in ("z", "row_max", "log_sum", "dz", "tokens", "entropy"):
        assert bwd(**{k: None}) == -1
    assert bwd(g_logp=None, g_entropy=None) == -1
    for k in ("z", "tokens", "row_max", "log_sum", "entropy", "g_logp", "g_entropy", "dz"):
        assert bwd(**{k: ODDER}) == -4
    assert bwd(T=0, z=None) == 0
