"""The projection with bias, activation and residual against its formulas in 64 bits: both paths, few and many tokens, odd sizes."""
import math

import pytest
import torch

from layer_util import act as act_of, gen, randn
from train_util import check, half_step

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _chain(n):
    # a sum of n products in fp32 (in blocks at least of 8 on the tensor cores, where an addition may be off by a whole step),
    # the bias, the activation (the hardware exponential and reciprocal: a few 2^-22)
    return n / 4 + 64


def _fma_chain(n):
    return n + 32


def _code(dtype):
    import transformer_rmsnorm_fwd_gb300 as L
    return L.LIGER_BF16 if dtype is BF else L.LIGER_F32


def fwd_case(dtype, T, H, N, act="gelu", bias=True, residual=True, keep=True, in_place=False, seed=0, X=None, W=None):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(seed)
    X = randn(g, T, H, dtype=dtype) if X is None else X
    W = randn(g, N, H, std=1.28 / math.sqrt(H), dtype=dtype) if W is None else W
    b = randn(g, N, std=0.5, dtype=dtype) if bias else None
    R = randn(g, T, N, dtype=dtype) if residual else None
    Y = R.clone() if in_place else torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    pre = torch.full((T, N), 7.0, dtype=torch.float16 if dtype is BF else F32, device="cuda") if keep else None
    L.liger_linear_act_fwd(X, W, Y, bias=b, residual=Y if in_place else R, act=act, pre=pre)
    p = X.double() @ W.double().T
    mag = X.double().abs() @ W.double().abs().T
    if bias:
        p, mag = p + b.double(), mag + b.double().abs()
    y, _ = act_of(act, p)
    c = _chain(H) if dtype is BF and H % 8 == 0 and N % 8 == 0 else _fma_chain(H)
    if keep:
        check(pre, p, mag, c, "pre")
    # every activation here has a slope of at most 1.13
    mag = 1.13 * mag
    if residual:
        y, mag = y + R.double(), mag + R.double().abs()
    check(Y, y, mag, c + 2, "Y")
    return Y, pre


SIZES = [(1, 64, 64), (1, 4096, 520), (2, 64, 256), (3, 128, 72), (5, 192, 1000), (8, 256, 128), (17, 320, 264), (33, 520, 1384),
         (64, 1024, 512), (65, 72, 4096), (100, 4096, 64), (128, 136, 640), (129, 512, 200), (200, 2048, 1024), (256, 256, 256),
         (257, 264, 776), (512, 64, 2048), (700, 1384, 520), (1111, 1384, 520), (2500, 200, 312)]


@pytest.mark.parametrize("T,H,N", SIZES)
def test_forward_bf16(cuda_lib, T, H, N):
    fwd_case(BF, T, H, N, act=ACTS[(T + H // 8 + N // 8) % 5], seed=T + H + N)


@pytest.mark.parametrize("T,H,N", [(1, 1, 1), (1, 7, 3), (2, 64, 9), (3, 65, 64), (4, 4096, 100), (31, 33, 35), (64, 64, 64), (65, 129, 63),
                                   (130, 257, 200), (300, 257, 1001), (513, 40, 8), (700, 1000, 30)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_odd_and_fp32(cuda_lib, dtype, T, H, N):
    fwd_case(dtype, T, H, N, act=ACTS[(T + H + N) % 5], seed=T + H + N)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [4, 150, 600])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("parts", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)])
def test_forward_parts(cuda_lib, dtype, T, act, parts):
    b, r, keep = parts
    fwd_case(dtype, T, 192, 136, act=act, bias=b, residual=r, keep=keep)


@pytest.mark.parametrize("dtype,T,H,N", [(BF, 3, 256, 264), (BF, 300, 256, 264), (BF, 90, 70, 33), (F32, 20, 48, 100)])
def test_residual_in_place_gives_the_same_bits(cuda_lib, dtype, T, H, N):
    a = fwd_case(dtype, T, H, N, act="silu", seed=4)
    b = fwd_case(dtype, T, H, N, act="silu", seed=4, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 5, 16, 17, 40, 128, 129, 1000])
def test_whole_numbers_come_out_exactly(cuda_lib, T):
    """Sums of small whole numbers are exact in fp32 in any order: every element of every tile is where it belongs."""
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(T)
    for dtype, H, N in ((BF, 136, 264), (BF, 64, 1032), (BF, 1032, 72), (F32, 77, 90), (BF, 33, 41)):
        X = torch.randint(-3, 4, (T, H), device="cuda", generator=g).to(dtype)
        W = torch.randint(-2, 3, (N, H), device="cuda", generator=g).to(dtype)
        b = torch.randint(-8, 9, (N,), device="cuda", generator=g).to(dtype)
        R = torch.randint(-8, 9, (T, N), device="cuda", generator=g).to(dtype)
        Y = torch.empty(T, N, dtype=dtype, device="cuda")
        L.liger_linear_act_fwd(X, W, Y, bias=b, residual=R, act="relu")
        p = X.double() @ W.double().T + b.double()
        assert torch.equal(Y, (p.clamp(min=0) + R.double()).to(dtype)), (dtype, H, N)
        dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty_like(b)
        dY = torch.randint(-3, 4, (T, N), device="cuda", generator=g).to(dtype)
        for act in ("none", "relu"):
            pre = p.to(torch.float16 if dtype is BF else F32)
            dp = dY.double() * ((pre.double() > 0).double() if act == "relu" else 1.0)
            ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, act, _code(dtype)), dtype=torch.uint8, device="cuda")
            for t in (dX, dW, db):
                t.fill_(7.0)
            L.liger_linear_act_bwd(dY, X, W, dX, dW, db, ws, pre=pre if act == "relu" else None, act=act)
            assert torch.equal(dX, (dp @ W.double()).to(dtype)) and torch.equal(dW, (dp.T @ X.double()).to(dtype)), (dtype, H, N)
            assert torch.equal(db, dp.sum(0).to(dtype))


def bwd_case(dtype, T, H, N, act="gelu", want=("dX", "dW", "db"), seed=0):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(seed)
    X, W = randn(g, T, H, dtype=dtype), randn(g, N, H, std=1.28 / math.sqrt(H), dtype=dtype)
    dY = randn(g, T, N, dtype=dtype)
    pre = randn(g, T, N, std=1.5, dtype=torch.float16 if dtype is BF else F32)
    out = {"dX": torch.full_like(X, 7.0), "dW": torch.full_like(W, 7.0), "db": torch.full((N,), 7.0, dtype=dtype, device="cuda")}
    out = {k: v if k in want else None for k, v in out.items()}
    need = L.liger_linear_act_bwd_workspace(T, H, N, act, _code(dtype))
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    L.liger_linear_act_bwd(dY, X if "dW" in want else X, W, out["dX"], out["dW"], out["db"], ws[:need],
                           pre=pre if act != "none" else None, act=act)
    assert bool((ws[need:] == 255).all())
    tc = dtype is BF and H % 8 == 0 and N % 8 == 0 and H >= 64 and N >= 64
    dp = dY.double() * act_of(act, pre.double())[1]
    # dP: its own arithmetic (a slope of magnitude up to 1.13, 32 roundings), and on the tensor cores one to bf16
    slack = 32 * 2.0 ** -24 * 1.13 * dY.double().abs() * (act != "none")
    err = slack + (half_step(BF) * dp.abs() if tc and act != "none" else 0)
    chain = _chain if tc else _fma_chain

    def held(got, ref, mag, extra, n, what):
        check(got, ref, mag + extra / (chain(n) * 2.0 ** -24), chain(n), what)

    if "dX" in want:
        held(out["dX"], dp @ W.double(), dp.abs() @ W.double().abs(), err @ W.double().abs(), N, "dX")
    if "dW" in want:
        held(out["dW"], dp.T @ X.double(), dp.abs().T @ X.double().abs(), err.T @ X.double().abs(), T, "dW")
    if "db" in want:
        check(out["db"], dp.sum(0), dp.abs().sum(0) + slack.sum(0) / ((T / 64 + 300) * 2.0 ** -24), T / 64 + 300, "db")
    return out


@pytest.mark.parametrize("T,H,N", SIZES)
def test_backward_bf16(cuda_lib, T, H, N):
    bwd_case(BF, T, H, N, act=ACTS[(T + H // 8 + N // 8) % 5], seed=T + H + N)


@pytest.mark.parametrize("T,H,N", [(1, 1, 1), (1, 7, 3), (3, 65, 64), (4, 1000, 100), (31, 33, 35), (65, 129, 63), (300, 257, 1001), (700, 100, 30)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_backward_odd_and_fp32(cuda_lib, dtype, T, H, N, act):
    bwd_case(dtype, T, H, N, act=act, seed=T + H + N)


@pytest.mark.parametrize("T,H,N", [(200, 200, 200), (17, 1600, 1999), (140, 2047, 131), (1024, 1024, 1001), (2000, 700, 300), (1599, 1601, 333),
                                   (2043, 101, 2000), (2048, 2048, 2047)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_fma_tiles_of_all_shapes(cuda_lib, dtype, T, H, N):
    """Products off the tensor cores large enough for each tile shape, with K split over clusters and whole."""
    if dtype is BF and H % 8 == 0 and N % 8 == 0:
        H += 1
    fwd_case(dtype, T, H, N, act="silu", seed=T)
    bwd_case(dtype, T, H, N, act="gelu_tanh", seed=T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("want", [("dX",), ("dW",), ("db",), ("dX", "db"), ("dX", "dW")])
def test_backward_parts(cuda_lib, dtype, act, want):
    bwd_case(dtype, 70, 192, 136, act=act, want=want)


@pytest.mark.parametrize("dtype,T,H,N", [(BF, 4, 128, 136), (BF, 200, 128, 136), (F32, 30, 24, 40)])
def test_saturated_activations(cuda_lib, dtype, T, H, N):
    """Sums far past the range of half precision: the kept value holds its sign, and the slopes are at their limits."""
    import transformer_rmsnorm_fwd_gb300 as L
    X = torch.full((T, H), 512.0, dtype=dtype, device="cuda")
    W = torch.full((N, H), 4.0, dtype=dtype, device="cuda")
    W[::2] *= -1
    dY = torch.ones(T, N, dtype=dtype, device="cuda")
    for act in ACTS[1:]:
        Y = torch.empty(T, N, dtype=dtype, device="cuda")
        pre = torch.empty(T, N, dtype=torch.float16 if dtype is BF else F32, device="cuda")
        L.liger_linear_act_fwd(X, W, Y, act=act, pre=pre)
        assert not Y[:, ::2].any() and bool((Y[:, 1::2] == 512.0 * 4 * H).all())
        assert bool((pre[:, 1::2] == min(512.0 * 4 * H, 65504.0 if dtype is BF else math.inf)).all())
        db, ws = torch.empty(N, dtype=dtype, device="cuda"), torch.empty(
            L.liger_linear_act_bwd_workspace(T, H, N, act, _code(dtype)), dtype=torch.uint8, device="cuda")
        L.liger_linear_act_bwd(dY, X, W, None, None, db, ws, pre=pre, act=act)
        assert not db[::2].any() and bool((db[1::2] == T).all())


@pytest.mark.parametrize("dtype,T,H,N", [(BF, 4, 128, 136), (BF, 300, 128, 264), (BF, 9, 33, 40), (F32, 70, 24, 40)])
def test_nan_stays_in_its_row_and_column(cuda_lib, dtype, T, H, N):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(8)
    X, W = randn(g, T, H, dtype=dtype), randn(g, N, H, dtype=dtype)
    X[T // 2, 3], W[5, H - 1] = float("nan"), float("nan")
    for act in ACTS:
        Y, pre = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, N, dtype=torch.float16 if dtype is BF else F32, device="cuda")
        L.liger_linear_act_fwd(X, W, Y, act=act, pre=pre)
        bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
        bad[T // 2], bad[:, 5] = True, True
        assert torch.equal(torch.isnan(Y), bad) and torch.equal(torch.isnan(pre), bad), act


@pytest.mark.parametrize("dtype,H,N", [(BF, 64, 72), (BF, 7, 9), (F32, 64, 72)])
def test_no_tokens(cuda_lib, dtype, H, N):
    import transformer_rmsnorm_fwd_gb300 as L
    X, W = torch.empty(0, H, dtype=dtype, device="cuda"), torch.ones(N, H, dtype=dtype, device="cuda")
    Y = torch.empty(0, N, dtype=dtype, device="cuda")
    L.liger_linear_act_fwd(X, W, Y)
    dW, db = torch.full_like(W, 7.0), torch.full((N,), 7.0, dtype=dtype, device="cuda")
    L.liger_linear_act_bwd(Y, X, W, X, dW, db, None)
    assert not dW.any() and not db.any()


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(cuda_lib, act):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(21)
    T, H, N = 5, 9, 6
    X, W, b, dY = (randn(g, *s) for s in ((T, H), (N, H), (N,), (T, N)))
    Y, pre = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty_like(b)
    ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, act, L.LIGER_F32), dtype=torch.uint8, device="cuda")
    L.liger_linear_act_fwd(X, W, Y, bias=b, act=act, pre=pre)
    L.liger_linear_act_bwd(dY, X, W, dX, dW, db, ws, pre=pre, act=act)

    def loss(X, W, b):
        return float((act_of(act, X.double() @ W.double().T + b.double())[0] * dY.double()).sum())

    for t, d, other in ((X, dX, lambda v: (v, W, b)), (W, dW, lambda v: (X, v, b)), (b, db, lambda v: (X, W, v))):
        for i in range(0, t.numel(), 3):
            up, down = t.double().clone(), t.double().clone()
            up.view(-1)[i] += 1e-6
            down.view(-1)[i] -= 1e-6
            diff = (loss(*other(up)) - loss(*other(down))) / 2e-6
            assert abs(diff - float(d.view(-1)[i])) < 3e-5 * (1 + abs(diff)), (act, i)


def test_refusals(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    X, W, Y = (torch.zeros(*s, dtype=BF, device="cuda") for s in ((4, 64), (72, 64), (4, 72)))
    for bad in (dict(X=X.t()), dict(W=W[:, :63]), dict(Y=Y.float()), dict(bias=W[0]), dict(residual=X), dict(act="tanh"),
                dict(pre=Y.clone()), dict(pre=Y.float()), dict(X=X.cpu()), dict(X=X.half(), W=W.half(), Y=Y.half())):
        a = dict(dict(X=X, W=W, Y=Y, bias=None, residual=None, act="none", pre=None), **bad)
        with pytest.raises((ValueError, TypeError)):
            L.liger_linear_act_fwd(a["X"], a["W"], a["Y"], bias=a["bias"], residual=a["residual"], act=a["act"], pre=a["pre"])
    buf = torch.zeros(4 * 64 + 8, dtype=BF, device="cuda")
    with pytest.raises(L.LigerError):           # not 16-byte aligned
        L.liger_linear_act_fwd(buf[4:4 + 256].view(4, 64), W, Y)
    with pytest.raises(L.LigerError):           # no workspace, and no kept values
        L.liger_linear_act_bwd(Y, X, W, X.clone(), None, None, None, pre=Y.half(), act="gelu")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(L.LigerError):
        L.liger_linear_act_bwd(Y, X, W, X.clone(), None, None, ws, act="gelu")
