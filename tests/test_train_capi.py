"""The C entry points of include/liger_train.h: all exported and bound, and their argument checks (host only: no CUDA call)."""
import ctypes
import os

import pytest

from transformer_rmsnorm_fwd_gb300 import _native, _train

OK, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        from transformer_rmsnorm_fwd_gb300 import build
        build.build()
    return _train._lib()


def test_exports_every_declared_function(lib):
    names = _train.header_functions()
    assert names and set(names) == set(_train.SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n
    import transformer_rmsnorm_fwd_gb300 as L
    for n in names:
        assert hasattr(L, n.replace("_async", "")), n


def _norm_fwd(lib, **kw):
    a = dict(z=OK, r=OK, w_post=OK, gate=OK, w_pre=OK, h=OK, y=OK, rz=OK, rh=OK, rows=6, cols=64, gates=1, a=1.0, b=1.0,
             eps=1e-6, dtype=1)
    a.update(kw)
    return lib.liger_block_norm_fwd(*a.values(), None)


def _norm_bwd(lib, **kw):
    a = dict(dh=OK, dy=OK, z=OK, h=OK, w_post=OK, gate=OK, w_pre=OK, rz=OK, rh=OK, dr=OK, dz=OK, dw_post=OK, dgate=OK,
             dw_pre=OK, ws=OK, ws_bytes=1 << 30, rows=6, cols=64, gates=1, a=1.0, b=1.0, dtype=1)
    a.update(kw)
    return lib.liger_block_norm_bwd(*a.values(), None)


def test_block_norm_fwd_checks(lib):
    assert _norm_fwd(lib, dtype=2) == -3
    assert _norm_fwd(lib, rows=-1) == -2 and _norm_fwd(lib, cols=0) == -2 and _norm_fwd(lib, gates=-1) == -2
    assert _norm_fwd(lib, gates=4) == -2                    # 6 rows
    assert _norm_fwd(lib, rows=1 << 46, cols=1 << 20) == -2
    assert _norm_fwd(lib, gates=0) == -1 and _norm_fwd(lib, gate=None) == -1
    assert _norm_fwd(lib, eps=-1.0) == -2 and _norm_fwd(lib, eps=float("nan")) == -2
    for k in ("z", "r", "h", "y"):
        assert _norm_fwd(lib, **{k: None}) == -1
    for k in ("z", "r", "h", "y", "w_post", "gate", "w_pre"):
        assert _norm_fwd(lib, **{k: ODD}) == -4
    assert _norm_fwd(lib, rows=0, z=None) == 0


def test_block_norm_bwd_checks(lib):
    assert _norm_bwd(lib, dtype=9) == -3 and _norm_bwd(lib, gates=5) == -2
    for k in ("dy", "z", "h", "rz", "rh", "dr", "dz", "dw_post", "dgate", "dw_pre"):
        assert _norm_bwd(lib, **{k: None}) == -1, k
    assert _norm_bwd(lib, w_pre=None, dh=None) == -1
    for k in ("dh", "dy", "z", "h", "dr", "dz", "dw_post", "dgate", "dw_pre"):
        assert _norm_bwd(lib, **{k: ODD}) == -4, k
    need = lib.liger_block_norm_bwd_workspace(6, 64, 1)
    assert need == 3 * 6 * 64 * 4 and lib.liger_block_norm_bwd_workspace(1 << 20, 64, 1) == 3 * 1024 * 64 * 4
    assert _norm_bwd(lib, ws_bytes=need - 1) == -6 and _norm_bwd(lib, ws=None) == -6 and _norm_bwd(lib, ws=ODD) == -6


def test_swiglu_ckpt8_checks(lib):
    for fn in (lib.liger_swiglu_fwd_ckpt8, lib.liger_swiglu_bwd_ckpt8):
        good = [OK] * 7
        assert fn(*good, 4, 64, 5, None) == -3
        assert fn(*good, 1 << 40, 1 << 20, 1, None) == -2
        assert fn(*good, -1, 64, 1, None) == -2 and fn(*good, 4, -64, 1, None) == -2
        assert fn(*([None] * 7), 0, 64, 1, None) == 0
        for k in range(7):
            assert fn(*[None if i == k else p for i, p in enumerate(good)], 4, 64, 1, None) == -1, k
    # codes and tensors want 16 bytes, scale bytes none
    for fn, wide in ((lib.liger_swiglu_fwd_ckpt8, (0, 1, 2, 3, 5)), (lib.liger_swiglu_bwd_ckpt8, (0, 1, 3, 5, 6))):
        for k in wide:
            assert fn(*[ODD if i == k else OK for i in range(7)], 4, 64, 1, None) == -4, k


def test_linear_swiglu_ckpt8_checks(lib):
    fwd = lambda *p, T=4, H=64, I=64, dt=1: lib.liger_fused_linear_swiglu_fwd_ckpt8(*p, T, H, I, dt, None)
    ps = [OK] * 8
    assert fwd(*ps, dt=0) == -3 and fwd(*ps, H=60) == -2 and fwd(*ps, I=12) == -2
    for k in range(8):
        assert fwd(*[None if i == k else OK for i in range(8)]) == -1, k
    for k in (0, 1, 2, 3, 4, 6):
        assert fwd(*[ODD if i == k else OK for i in range(8)]) == -4, k
    need = lib.liger_fused_linear_swiglu_workspace(4, 64)
    bwd = lambda *p, ws=OK, n=need, dt=1: lib.liger_fused_linear_swiglu_bwd_ckpt8(*p, ws, n, 4, 64, 64, dt, None)
    ps = [OK] * 11
    assert bwd(*ps, dt=0) == -3 and bwd(*ps, n=need - 1) == -6 and bwd(*ps, ws=None) == -6
    for k in range(11):
        assert bwd(*[None if i == k else OK for i in range(11)]) == -1, k
    for k in (0, 1, 2, 3, 4, 6, 8, 9, 10):
        assert bwd(*[ODD if i == k else OK for i in range(11)]) == -4, k


def _logp(fn, **kw):
    a = dict(X=OK, W=OK, labels=OK, T=4, H=64, V=300, ign=-100, logp=OK, ws=OK, n=1 << 30, dtype=1)
    a.update(kw)
    return fn(*a.values(), None)


def _policy(fn, **kw):
    a = dict(X=OK, W=OK, labels=OK, cu=OK, old=OK, ref=OK, adv=OK, T=4, H=64, V=300, B=2, ign=-100, reduction=0, flags=0,
             lo=0.2, hi=0.2, beta=0.1, gs=1.0, loss=OK, stats=OK, logp=OK, dX=OK, dW=OK, ws=OK, n=1 << 40, chunk=0, dtype=1)
    a.update(kw)
    return fn(*a.values(), None)


def test_logp_checks(lib):
    for fn in (lib.liger_linear_logp_fwd, lib.liger_linear_logp_fwd_async):
        assert _logp(fn, dtype=3) == -3 and _logp(fn, T=-1) == -2 and _logp(fn, V=0) == -2 and _logp(fn, H=0) == -2
        assert _logp(fn, V=5000000, dtype=0) == -2 and _logp(fn, T=1 << 23, V=2, dtype=0) == -2
        assert _logp(fn, T=1 << 31) == -2 and _logp(fn, T=0, X=None) == 0
        for k in ("X", "W", "labels", "logp"):
            assert _logp(fn, **{k: None}) == -1, k
        for k in ("X", "W"):
            assert _logp(fn, **{k: ODD}) == -4, k
        assert _logp(fn, labels=ctypes.c_void_p(0x1004)) == -4 and _logp(fn, logp=ctypes.c_void_p(0x1002)) == -4
        need = lib.liger_linear_logp_workspace(4, 64, 300, 1)
        assert need > 0 and _logp(fn, n=need - 1) == -6 and _logp(fn, ws=None) == -6 and _logp(fn, ws=ODD) == -6
    assert lib.liger_linear_logp_workspace(4, 64, 300, 9) == 0 and lib.liger_linear_logp_workspace(-1, 64, 300, 1) == 0


def test_policy_checks(lib):
    nan = float("nan")
    for fn in (lib.liger_linear_policy_fwd_bwd, lib.liger_linear_policy_fwd_bwd_async):
        assert _policy(fn, dtype=3) == -3
        for kw in (dict(T=-1), dict(H=0), dict(V=0), dict(B=0), dict(chunk=-1), dict(reduction=3), dict(reduction=-1),
                   dict(flags=2), dict(lo=-0.1), dict(lo=1.1), dict(hi=-0.1), dict(lo=nan), dict(hi=nan), dict(beta=nan),
                   dict(gs=nan), dict(T=1 << 31), dict(V=5000000, dtype=0), dict(T=1 << 23, V=2, dtype=0)):
            assert _policy(fn, **kw) == -2, kw
        for k in ("X", "W", "labels", "cu", "old", "ref", "adv", "loss"):
            assert _policy(fn, **{k: None}) == -1, k
        for k in ("X", "W", "dX", "dW"):
            assert _policy(fn, **{k: ODD}) == -4, k
        for k in ("cu", "old", "ref", "adv", "loss", "stats", "logp"):
            assert _policy(fn, **{k: ctypes.c_void_p(0x1002)}) == -4, k
        need = lib.liger_linear_policy_workspace(4, 64, 300, 2, 0, 1)
        assert need > 0 and _policy(fn, n=need - 1) == -6 and _policy(fn, ws=None) == -6 and _policy(fn, ws=ODD) == -6
    assert lib.liger_linear_policy_workspace(4, 64, 300, 0, 0, 1) == 0


def test_policy_logp_is_no_input(lib):
    """logp over old_logp, ref_logp or adv would be read back as the policy's own: refused."""
    at = lambda n: ctypes.c_void_p(0x100000 + n)
    for fn in (lib.liger_linear_policy_fwd_bwd, lib.liger_linear_policy_fwd_bwd_async):
        for kw in (dict(old=at(0)), dict(ref=at(0)), dict(adv=at(0)), dict(old=at(12)), dict(ref=at(-12)), dict(adv=at(-4)),
                   dict(adv=at(-12), flags=1)):
            assert _policy(fn, logp=at(0), **kw) == -2, kw


def test_nothing_is_allocated_or_thrown():
    """The library allocates nothing, and no exception can leave a C entry: no owning std types, new or throw in its sources."""
    import glob
    import re
    src = os.path.join(_native.PKG, "csrc")
    for f in glob.glob(os.path.join(src, "*.cu")) + glob.glob(os.path.join(src, "*.cuh")):
        with open(f) as h:
            text = re.sub(r"//[^\n]*", "", h.read())
        found = re.findall(r"std::(?:function|vector|string|map|unordered_map|deque|unique_ptr|shared_ptr)\b|\bnew\s+\w|\bthrow\b", text)
        assert not found, (os.path.basename(f), found)
