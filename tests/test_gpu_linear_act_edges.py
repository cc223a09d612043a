"""The projection's activations at the edges of their types: sums near 0, where half precision ends."""
import pytest
import torch

from layer_util import act as act_of, gen, randn
from train_util import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# few tokens and 128-feature tiles, tiles of CTA pairs (96 of them), fp32 FMA for bf16 and for fp32
PATHS = [(BF, 4, 64, 72), (BF, 300, 128, 264), (BF, 3000, 64, 2048), (BF, 9, 33, 40), (BF, 200, 70, 90), (F32, 30, 24, 40)]


def code(dtype):
    import transformer_rmsnorm_fwd_gb300 as L
    return L.LIGER_BF16 if dtype is BF else L.LIGER_F32


def small_sums(g, dtype, T, H, N):
    """X with one power of two (2^-100 to 2^-20, the same in every row that has it at h) a row and W of small whole numbers: every
    sum is that power times one of them, exactly."""
    at = torch.arange(T, device="cuda") % H
    power = 2.0 ** torch.randint(-100, -19, (H,), device="cuda", generator=g).double()
    X = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    X[torch.arange(T, device="cuda"), at] = power[at]
    W = torch.randint(-3, 4, (N, H), device="cuda", generator=g).to(dtype)
    return X.to(dtype), W


@pytest.mark.parametrize("dtype,T,H,N", PATHS)
def test_relu_of_tiny_sums_keeps_its_gradient(cuda_lib, dtype, T, H, N):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(T + N)
    X, W = small_sums(g, dtype, T, H, N)
    p = X.double() @ W.double().T
    Y, pre = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, N, dtype=torch.float16 if dtype is BF else F32, device="cuda")
    L.liger_linear_act_fwd(X, W, Y, act="relu", pre=pre)
    assert torch.equal(Y, p.clamp(min=0).to(dtype))
    assert torch.equal(pre > 0, p > 0) and not bool(torch.isnan(pre).any())
    dY = torch.randint(-3, 4, (T, N), device="cuda", generator=g).to(dtype)
    dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty(N, dtype=dtype, device="cuda")
    ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, "relu", code(dtype)), dtype=torch.uint8, device="cuda")
    L.liger_linear_act_bwd(dY, X, W, dX, dW, db, ws, pre=pre, act="relu")
    dp = dY.double() * (p > 0)
    # whole numbers, and whole numbers times one power of two: exact before the one rounding
    assert torch.equal(dX, (dp @ W.double()).to(dtype)) and torch.equal(db, dp.sum(0).to(dtype))
    assert torch.equal(dW, (dp.T @ X.double()).to(dtype)) and bool(dW.any())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,T,H,N", PATHS)
def test_smooth_activations_of_tiny_sums(cuda_lib, dtype, T, H, N, act):
    """The value kept for a sum below 2^-14 is at most 2^-25 off, and with slopes' derivatives of at most 1 so is the slope: of one
    half, 2^-24 of it beside the 32 roundings of its arithmetic."""
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(T + N + 1)
    X, W = small_sums(g, dtype, T, H, N)
    Y, pre = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, N, dtype=torch.float16 if dtype is BF else F32, device="cuda")
    L.liger_linear_act_fwd(X, W, Y, act=act, pre=pre)
    dY, db = randn(g, T, N, dtype=dtype), torch.empty(N, dtype=dtype, device="cuda")
    ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, act, code(dtype)), dtype=torch.uint8, device="cuda")
    L.liger_linear_act_bwd(dY, X, W, None, None, db, ws, pre=pre, act=act)
    dp = dY.double() * act_of(act, X.double() @ W.double().T)[1]
    check(db, dp.sum(0), dp.abs().sum(0), T / 64 + 300 + 34, "db")


def far_points(n):
    """n values of bf16 over [-12, 12], close together near 0 too."""
    half = n // 2
    p = torch.cat((torch.linspace(-12, 12, n - half, dtype=torch.float64), 12 * torch.linspace(-1, 1, half, dtype=torch.float64) ** 5))
    return p.to(BF).double().cuda()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,T,H,N", [(BF, 1, 64, 4000), (BF, 300, 128, 2000), (BF, 3000, 64, 2048), (BF, 3, 33, 1001), (F32, 5, 24, 2000)])
def test_activations_of_far_sums_relative_to_themselves(cuda_lib, dtype, T, H, N, act):
    """A result that is small because its activation is (p far below 0) has its type's relative error.  Before the rounding to it
    the exponent of e, at most 88 in fp32's range, is off by up to 4 roundings of its size, and there are up to 40 of the result's:
    400 of 2^-24.  The hardware's functions leave out what is below 2^-126, here times 12."""
    import transformer_rmsnorm_fwd_gb300 as L
    p = far_points(N)
    X, W = torch.zeros(T, H, dtype=dtype, device="cuda"), torch.zeros(N, H, dtype=dtype, device="cuda")
    X[:, 0], W[:, 0] = 1.0, p.to(dtype)
    Y, pre = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, N, dtype=torch.float16 if dtype is BF else F32, device="cuda")
    L.liger_linear_act_fwd(X, W, Y, act=act, pre=pre)
    y, s = act_of(act, p)
    u = torch.finfo(dtype).eps / 2
    rel = 400 * 2.0 ** -24
    assert bool(((Y.double() - y).abs() <= (u + rel) * y.abs() + 2.0 ** -122).all())
    # one row's slope comes out as db; its two terms may cancel
    dY, db = torch.ones(1, N, dtype=dtype, device="cuda"), torch.empty(N, dtype=dtype, device="cuda")
    ws = torch.empty(L.liger_linear_act_bwd_workspace(1, H, N, act, code(dtype)) + 256, dtype=torch.uint8, device="cuda")
    L.liger_linear_act_bwd(dY, X[:1].contiguous(), W, None, None, db, ws, pre=pre[:1].contiguous(), act=act)
    value = y / torch.where(p == 0, 1.0, p)
    terms = value.abs() + (s - value).abs()
    # (a sum below 2^-14 was kept in steps of 2^-24; what the functions leave out below 2^-126 counts p times the derivative of the
    # exponent here, in gelu with tanh at 12: 12 (1.596 + 0.2141 * 144) = 389 < 2^9)
    floor = 2.0 ** -24 * (p.abs() < 2.0 ** -14) + 2.0 ** -117
    assert bool(((db.double() - s).abs() <= u * s.abs() + rel * terms + floor).all())


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T,H,N", [(4, 64, 72), (300, 128, 264), (3000, 64, 2048), (9, 33, 40), (200, 70, 90)])
def test_sums_that_overflow_keep_their_limits_slope(cuda_lib, T, H, N, act):
    """Infinite sums of bf16 tensors are kept as half precision's largest, where every slope is 0 or 1."""
    import transformer_rmsnorm_fwd_gb300 as L
    X, W = torch.full((T, H), 1e30, dtype=BF, device="cuda"), torch.full((N, H), 1e30, dtype=BF, device="cuda")
    W[::2] *= -1
    Y, pre = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, N, dtype=torch.float16, device="cuda")
    L.liger_linear_act_fwd(X, W, Y, act=act, pre=pre)
    assert bool((Y[:, 1::2] == float("inf")).all())
    assert bool((pre[:, 1::2] == 65504.0).all()) and bool((pre[:, ::2] == -65504.0).all())
    dY, db = torch.ones(T, N, dtype=BF, device="cuda"), torch.empty(N, dtype=BF, device="cuda")
    ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, act), dtype=torch.uint8, device="cuda")
    L.liger_linear_act_bwd(dY, X, W, None, None, db, ws, pre=pre, act=act)
    assert not db[::2].any() and bool((db[1::2] == torch.tensor(T, dtype=BF)).all())
