"""The post-training operators right behind a kernel that lets its successor start before it has written anything: each
input in turn, of each call, is written by such a kernel only, into a buffer that held other values."""
import ctypes
import os
import subprocess

import pytest
import torch

from transformer_rmsnorm_fwd_gb300 import build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as lib
    return lib


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("native") / "early_producer.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "early_producer.cu")
    p = subprocess.run([build.nvcc(), *build._flags(False), "-shared", "-o", out, src], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    lib = ctypes.CDLL(out)
    lib.late_copy_launch.argtypes = [ctypes.c_void_p] * 2 + [ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p]

    def copy(dst, src):
        assert dst.is_contiguous() and src.is_contiguous() and dst.nbytes == src.nbytes
        rc = lib.late_copy_launch(dst.data_ptr(), src.data_ptr(), dst.nbytes, 30000, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
    return copy


def _stale(t):
    """Values that a call can read without harm, and that change its results."""
    if t.dtype == torch.int64:
        return torch.where(t == -100, t, t.flip(0).clamp(min=0))
    if t.dtype == torch.int32:
        return t.clone().fill_(0)
    if t.dtype in (torch.int8, torch.uint8):
        return t.flip(0).contiguous()
    return torch.full_like(t, 0.75)


def _cases(L, spaces):
    """name, inputs, outputs, call; every workspace goes into `spaces`"""
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*s, dt=BF, std=1.0):
        return (torch.randn(*s, device="cuda", generator=g) * std).to(dt)

    def empty(n):
        spaces.append(torch.empty(max(n, 256), dtype=torch.uint8, device="cuda"))
        return spaces[-1]

    def norms(rows, cols, dt):
        i = dict(z=rnd(rows, cols, dt=dt), r=rnd(rows, cols, dt=dt), wp=rnd(cols, dt=dt), g=rnd(1, cols, dt=dt), wn=rnd(cols, dt=dt))
        o = dict(h=torch.empty_like(i["z"]), y=torch.empty_like(i["z"]), rz=torch.empty(rows, device="cuda"),
                 rh=torch.empty(rows, device="cuda"))
        yield f"norms_fwd {rows}x{cols} {dt}", i, o, lambda i=i, o=o: L.liger_block_norm_fwd(
            i["z"], i["r"], o["h"], o["y"], i["wp"], i["g"], i["wn"], o["rz"], o["rh"])
        b = dict(dh=rnd(rows, cols, dt=dt), dy=rnd(rows, cols, dt=dt), z=i["z"].clone(), h=rnd(rows, cols, dt=dt), wp=i["wp"].clone(),
                 g=i["g"].clone(), wn=i["wn"].clone(), rz=rnd(rows, dt=torch.float32).abs(), rh=rnd(rows, dt=torch.float32).abs())
        p = dict(dr=torch.empty_like(i["z"]), dz=torch.empty_like(i["z"]), dwp=torch.empty_like(i["wp"]), dg=torch.empty_like(i["g"]),
                 dwn=torch.empty_like(i["wn"]))
        ws = empty(L.liger_block_norm_bwd_workspace(rows, cols, 1))
        yield f"norms_bwd {rows}x{cols} {dt}", b, p, lambda b=b, p=p, ws=ws: L.liger_block_norm_bwd(
            b["dh"], b["dy"], b["z"], b["h"], p["dr"], p["dz"], ws, b["wp"], b["g"], b["wn"], b["rz"], b["rh"], p["dwp"], p["dg"],
            p["dwn"])

    def swiglu(rows, cols, dt):
        i = dict(g=rnd(rows, cols, dt=dt), u=rnd(rows, cols, dt=dt))
        kept = (*L.liger_ckpt8_empty(rows, cols), *L.liger_ckpt8_empty(rows, cols))
        y = torch.empty_like(i["g"])
        yield (f"swiglu_fwd {rows}x{cols} {dt}", i, dict(zip(("y", "g8", "gs", "u8", "us"), (y, *kept))),
               lambda i=i, y=y, kept=kept: L.liger_swiglu_fwd_ckpt8(i["g"], i["u"], y, *kept))
        k = (*L.liger_ckpt8_empty(rows, cols), *L.liger_ckpt8_empty(rows, cols))
        L.liger_swiglu_fwd_ckpt8(i["g"], i["u"], y, *k)
        b = dict(dy=rnd(rows, cols, dt=dt), g8=k[0], gs=k[1], u8=k[2], us=k[3])
        o = dict(dg=torch.empty_like(y), du=torch.empty_like(y))
        yield (f"swiglu_bwd {rows}x{cols} {dt}", b, o, lambda b=b, o=o: L.liger_swiglu_bwd_ckpt8(
            b["dy"], b["g8"], b["gs"], b["u8"], b["us"], o["dg"], o["du"]))

    def mlp(T, H, I):
        i = dict(X=rnd(T, H), Wg=rnd(I, H, std=H ** -0.5), Wu=rnd(I, H, std=H ** -0.5))
        kept = (*L.liger_ckpt8_empty(T, I), *L.liger_ckpt8_empty(T, I))
        out = torch.empty(T, I, device="cuda", dtype=BF)
        yield (f"linear_swiglu_fwd {T}", i, dict(zip(("out", "g8", "gs", "u8", "us"), (out, *kept))),
               lambda: L.liger_fused_linear_swiglu_fwd_ckpt8(i["X"], i["Wg"], i["Wu"], out, *kept))
        k = (*L.liger_ckpt8_empty(T, I), *L.liger_ckpt8_empty(T, I))
        L.liger_fused_linear_swiglu_fwd_ckpt8(i["X"], i["Wg"], i["Wu"], out, *k)
        b = dict(X=i["X"].clone(), Wg=i["Wg"].clone(), Wu=i["Wu"].clone(), dH=rnd(T, I), g8=k[0], gs=k[1], u8=k[2], us=k[3])
        o = dict(dX=torch.empty_like(i["X"]), dWg=torch.empty_like(i["Wg"]), dWu=torch.empty_like(i["Wu"]))
        ws = empty(L.liger_fused_linear_swiglu_workspace(T, I))
        yield (f"linear_swiglu_bwd {T}", b, o, lambda: L.liger_fused_linear_swiglu_bwd_ckpt8(
            b["X"], b["Wg"], b["Wu"], b["dH"], b["g8"], b["gs"], b["u8"], b["us"], o["dX"], o["dWg"], o["dWu"], ws))

    def head(T, H, V, dt, wait):
        code = L.LIGER_BF16 if dt is BF else L.LIGER_F32
        lab = torch.randint(0, V, (T,), device="cuda", generator=g)
        lab[::5] = -100
        i = dict(X=rnd(T, H, dt=dt), W=rnd(V, H, dt=dt, std=H ** -0.5), lab=lab)
        o = dict(logp=torch.empty(T, device="cuda"))
        ws = empty(L.liger_linear_logp_workspace(T, H, V, code))
        yield (f"logp {T} {dt} {wait}", i, o, lambda: L.liger_linear_logp_fwd(i["X"], i["W"], i["lab"], o["logp"], ws, wait=wait))
        b = dict(X=i["X"].clone(), W=i["W"].clone(), lab=lab.clone(), old=rnd(T, dt=torch.float32) - 7, ref=rnd(T, dt=torch.float32) - 7,
                 adv=rnd(1, dt=torch.float32))
        p = dict(loss=torch.empty(1, device="cuda"), dX=torch.empty_like(i["X"]), dW=torch.empty_like(i["W"]),
                 stats=torch.empty(2, device="cuda"), logp=torch.empty(T, device="cuda"))
        pws = empty(L.liger_linear_policy_workspace(T, H, V, 1, 0, code))
        yield (f"policy {T} {dt} {wait}", b, p, lambda: L.liger_linear_policy_fwd_bwd(
            b["X"], b["W"], b["lab"], b["old"], b["adv"], p["loss"], p["dX"], p["dW"], pws, ref_logp=b["ref"], logp=p["logp"],
            stats=p["stats"], beta=0.1, wait=wait))
    for rows, cols, dt in ((4, 1024, BF), (400, 1024, BF), (400, 1001, torch.float32), (40, 37, BF), (200, 8192, BF)):
        yield from norms(rows, cols, dt)
    for rows, cols, dt in ((200, 1024, BF), (100, 520, BF), (100, 33, torch.float32)):
        yield from swiglu(rows, cols, dt)
    for T in (70, 700):
        yield from mlp(T, 256, 544)
    for T, H, V, dt in ((1, 256, 2000, BF), (300, 256, 2000, BF), (700, 256, 2000, BF), (60, 64, 300, torch.float32)):
        for wait in (True, False):
            yield from head(T, H, V, dt, wait)


def test_inputs_written_late_by_the_kernel_before(L, late):
    """The results are the same bits as with inputs that stood there long before, and none is left from the stale values."""
    spaces = []
    for name, inputs, outputs, call in _cases(L, spaces):
        def clear():
            for v in spaces:
                v.fill_(255)
            del spaces[:-1]
            for v in outputs.values():
                v.fill_(0x55 if v.dtype in (torch.int8, torch.uint8) else float("nan"))
        clear()
        call()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in outputs.items()}
        for key, t in inputs.items():
            fresh, stale = t.clone(), _stale(t)
            for _ in range(3):
                t.copy_(stale)
                clear()
                torch.cuda.synchronize()
                late(t, fresh)
                call()
                torch.cuda.synchronize()
                for k, v in outputs.items():
                    same = torch.equal(v.view(torch.uint8), want[k].view(torch.uint8))
                    assert same, (name, key, k)
