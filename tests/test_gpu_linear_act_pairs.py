"""The projection on tiles of CTA pairs against its formulas in 64 bits: every activation with bias, residual and kept sums, ragged
last tiles, dW with its last round split along the tokens and whole; and which kernels the sizes of these tests run."""
import ctypes

import pytest
import torch

from layer_util import gen
from test_gpu_linear_act import ACTS, BF, bwd_case, fwd_case

pytestmark = pytest.mark.gpu
# 90 tiles forward, 72 of dX, 80 of dW: on 76 pairs 4 of them are left for a last round, in 2 ranges of the tokens
RAGGED = (2056, 2040, 2552)
# X of more than 32 MiB, whose columns dW takes in groups; 14 tiles of a last round, in 5 ranges
GROUPED = (8200, 2056, 2552)


class KernelNode(ctypes.Structure):     # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 7), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def kernels(fn):
    """Names, as they are mangled, of the kernels that fn launches on its stream: captured, and read from the graph's nodes."""
    cu = ctypes.CDLL("libcuda.so.1")

    def call(name, *args):
        rc = getattr(cu, name)(*args)
        assert rc == 0, (name, rc)

    fn()
    torch.cuda.synchronize()
    stream, graph, n, names = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t(), set()
    with torch.cuda.stream(stream):
        call("cuStreamBeginCapture_v2", ctypes.c_void_p(stream.cuda_stream), 2)     # relaxed
        try:
            fn()
        finally:
            call("cuStreamEndCapture", ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph))
    call("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    call("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    for node in nodes:
        kind, k, name = ctypes.c_int(), KernelNode(), ctypes.c_char_p()
        call("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value == 0:
            call("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(k))
            if k.func:
                call("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(k.func))
            else:
                call("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(k.kern))
            names.add(name.value.decode())
    call("cuGraphDestroy", graph)
    return names


def calls(dtype, T, H, N, act="gelu", dX=True):
    import transformer_rmsnorm_fwd_gb300 as L
    X, W, dY = (torch.zeros(*s, dtype=dtype, device="cuda") for s in ((T, H), (N, H), (T, N)))
    Y, pre, b = torch.empty_like(dY), torch.empty(T, N, dtype=torch.float16 if dtype is BF else dtype, device="cuda"), torch.zeros(
        N, dtype=dtype, device="cuda")
    out = (torch.empty_like(X) if dX else None, torch.empty_like(W), torch.empty_like(b))
    code = L.LIGER_BF16 if dtype is BF else L.LIGER_F32
    ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, act, code) + 256, dtype=torch.uint8, device="cuda")

    def fn():
        L.liger_linear_act_fwd(X, W, Y, bias=b, residual=dY, act=act, pre=pre)
        L.liger_linear_act_bwd(dY, X, W, *out, ws, pre=pre, act=act)
    return fn


FWD, STORE, WHOLE, SPLIT = (f"tc_gemm_kernelILi{a}ELi{b}ELi{e}ELi1ELi{m}EE" for a, b, e, m in ((0, 0, 8, 0), (0, 1, 1, 0), (1, 1, 2, 0), (1, 1, 2, 2)))


def test_these_sizes_run_every_path(cuda_lib):
    """A threshold that moves would leave a path without a test of its values: then other sizes are to be taken here."""
    def has(names, part):
        return any(part in n for n in names)
    for size in (RAGGED, GROUPED):
        names = kernels(calls(BF, *size))
        assert all(has(names, k) for k in (FWD, STORE, SPLIT, "split_join", "linear_db")), (size, names)
        assert not has(names, "linear_small"), (size, names)
        names = kernels(calls(BF, *size, dX=False))
        assert has(names, WHOLE) and not has(names, SPLIT) and not has(names, "split_join"), (size, names)
    names = kernels(calls(BF, 70, 192, 136))
    assert all(has(names, f"linear_smallILi{a}ELi{b}EE") for a, b in ((0, 0), (1, 0), (1, 1))) and not has(names, "tc_gemm_kernel"), names
    assert has(kernels(calls(BF, 70, 190, 136)), "fma_gemm")
    assert has(kernels(calls(torch.float32, 70, 192, 136)), "fma_gemm")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("parts", [(True, True, True), (False, True, False), (True, False, True)])
def test_forward_pairs(cuda_lib, act, parts):
    b, r, keep = parts
    fwd_case(BF, *RAGGED, act=act, bias=b, residual=r, keep=keep, seed=len(act))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_forward_pairs_in_place_gives_the_same_bits(cuda_lib, act):
    a, b = (fwd_case(BF, *RAGGED, act=act, seed=5, in_place=p) for p in (False, True))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("want", [("dX", "dW", "db"), ("dW", "db"), ("dX",)])
def test_backward_pairs(cuda_lib, act, want):
    bwd_case(BF, *RAGGED, act=act, want=want, seed=len(act) + len(want))


@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_large_inputs(cuda_lib, act):
    fwd_case(BF, *GROUPED, act=act, seed=1)
    for want in (("dX", "dW", "db"), ("dW",)):
        bwd_case(BF, *GROUPED, act=act, want=want, seed=2)


@pytest.mark.parametrize("T,H,N", [RAGGED, (2300, 1800, 2304), (300, 2048, 8200)])
def test_whole_numbers_come_out_exactly_on_pairs(cuda_lib, T, H, N):
    """Sums of small whole numbers are exact in fp32 in any order: every element of every tile and split is where it belongs."""
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(T)
    X = torch.randint(-3, 4, (T, H), device="cuda", generator=g).to(BF)
    W = torch.randint(-2, 3, (N, H), device="cuda", generator=g).to(BF)
    b, R = (torch.randint(-8, 9, s, device="cuda", generator=g).to(BF) for s in ((N,), (T, N)))
    dY = torch.randint(-3, 4, (T, N), device="cuda", generator=g).to(BF)
    p = X.double() @ W.double().T + b.double()
    for act in ("none", "relu"):
        Y, pre = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, N, dtype=torch.float16, device="cuda")
        L.liger_linear_act_fwd(X, W, Y, bias=b, residual=R, act=act, pre=pre)
        assert torch.equal(Y, ((p.clamp(min=0) if act == "relu" else p) + R.double()).to(BF))
        assert torch.equal(pre, p.to(torch.float16))
        dp = dY.double() * ((p > 0).double() if act == "relu" else 1.0)
        ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, act), dtype=torch.uint8, device="cuda")
        for with_dx in (True, False):
            dX, dW, db = (torch.full_like(t, 7.0) for t in (X, W, b))
            L.liger_linear_act_bwd(dY, X, W, dX if with_dx else None, dW, db, ws, pre=pre, act=act)
            assert torch.equal(dW, (dp.T @ X.double()).to(BF)) and torch.equal(db, dp.sum(0).to(BF))
            assert torch.equal(dX, (dp @ W.double()).to(BF)) if with_dx else bool((dX == 7.0).all())


def test_results_repeat_bit_for_bit(cuda_lib):
    for size in (RAGGED, (8200, 1024, 2048)):
        a, b = (fwd_case(BF, *size, act="gelu", seed=9) for _ in range(2))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = (bwd_case(BF, *size, act="gelu", seed=9) for _ in range(2))
        assert all(torch.equal(a[k], b[k]) for k in a)
