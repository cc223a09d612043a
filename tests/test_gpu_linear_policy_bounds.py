"""The policy loss and the log-probabilities within the bounds of policy_bounds, under which a k range, a token block or a
rounding that does not belong shows (test_policy_bounds plants these): every split of dX, both forms, compacted tokens."""
import pytest
import torch

from policy_bounds import Gradients, logit_bounds, logp_bounds, signed_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as lib
    return lib


def _kind(T, dt):
    return "fp32" if dt is torch.float32 else "few" if T <= 4 else "tc"


@pytest.mark.parametrize("wait", [True, False])
@pytest.mark.parametrize("T,H,V,masked,chunk", [
    (2600, 2048, 66536, 0.0, 0),   # a full round of dX tiles and 12 split ones, over two slabs of the vocabulary
    (2600, 2048, 3000, 0.0, 0),    # the same in one launch
    (20, 4096, 70000, 0.0, 0),     # 16 tiles split over all pairs
    (130, 520, 2100, 0.0, 0),      # 3 tiles; k ranges that do not divide the k-blocks
    (900, 1024, 20000, 0.5, 0),    # compacted (in the waiting form)
    (700, 256, 3000, 0.1, 0),
    (700, 256, 3000, 0.0, 128),  # several chunks: dW summed in fp32 between them
])
def test_gradients(L, T, H, V, masked, chunk, wait):
    X, W, labels, rest = signed_inputs(T, H, V, T + V, "cuda", masked)
    at = torch.nonzero(labels != -100)[:, 0]
    n = len(at)
    z, e = logit_bounds(X[at], W, "tc")
    lp, *_ = logp_bounds(z, e, labels[at])
    old = torch.full((T,), float("nan"), device="cuda")
    old[at] = (lp - 0.1).float()                        # a ratio of 1.1: inside the clip range, all of one sign
    c = torch.exp(lp - old[at].double()) / n
    G = Gradients(X[at], W, labels[at], c, z, e, spread=T / n)
    del z, e
    loss, logp = torch.empty(1, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.full_like(X, 7.0), torch.full_like(W, 7.0)
    ws = torch.full((L.liger_linear_policy_workspace(T, H, V, 1, chunk),), 255, dtype=torch.uint8, device="cuda")
    L.liger_linear_policy_fwd_bwd(X, W, labels, old, torch.ones(1, device="cuda"), loss, dX, dW, ws, logp=logp, chunk=chunk,
                                  wait=wait)
    assert bool(((logp[at].double() - G.lp).abs() <= G.e_lp).all())
    assert abs(float(loss) + float(c.sum())) <= float((c * G.e_c).sum()) + 2 ** -22 * float(c.sum())
    want, bound = G.dX()
    over = (dX[at].double() - want).abs() - bound
    assert bool((over <= 0).all()), (int((over > 0).sum()), float(over.max()))
    assert bool((dX[labels == -100] == 0).all())
    del want, bound, over
    for a in range(0, V, 16384):
        rows = slice(a, min(V, a + 16384))
        want, bound = G.dW(rows)
        over = (dW[rows].double() - want).abs() - bound
        assert bool((over <= 0).all()), (a, int((over > 0).sum()), float(over.max()))


@pytest.mark.parametrize("wait", [True, False])
@pytest.mark.parametrize("T,H,V,dt", [(1, 4096, 5001, "bf16"), (4, 4096, 5001, "bf16"), (3, 1024, 20000, "bf16"),
                                      (5, 4096, 5001, "bf16"), (40, 4096, 20000, "bf16"), (600, 2048, 3000, "bf16"),
                                      (1, 512, 3000, "f32"), (90, 1000, 2000, "f32"), (300, 256, 1024, "f32")])
def test_logp(L, T, H, V, dt, wait):
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(T + H)
    X = torch.randn(T, H, device="cuda", generator=g).to(dtype)
    W = (torch.randn(V, H, device="cuda", generator=g) * 1.3 * H ** -0.5).to(dtype)
    labels = torch.randint(0, V, (T,), device="cuda", generator=g)
    z, e = logit_bounds(X, W, _kind(T, dtype))
    lp, bound, *_ = logp_bounds(z, e, labels)
    ws = torch.empty(L.liger_linear_logp_workspace(T, H, V, L.LIGER_BF16 if dt == "bf16" else L.LIGER_F32), dtype=torch.uint8,
                     device="cuda")
    logp = torch.full((T,), 7.0, device="cuda")
    L.liger_linear_logp_fwd(X, W, labels, logp, ws, wait=wait)
    assert bool(((logp.double() - lp).abs() <= bound).all())
