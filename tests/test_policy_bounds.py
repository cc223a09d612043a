"""The bounds of policy_bounds reject wrong results: mistakes planted in the 64-bit form lie further from it than twice the
bound, so that a kernel that made them could not pass.  On the CPU."""
import pytest
import torch

from policy_bounds import Gradients, logit_bounds, logp_bounds, signed_inputs


def _rejected(wrong, right, bound):
    """The share of elements that are too far off."""
    return float(((wrong - right).abs() > 2 * bound).double().mean())


def _model(T, H, V, seed):
    X, W, labels, rest = signed_inputs(T, H, V, seed, "cpu")
    z, e = logit_bounds(X, W, "tc")
    c = torch.full((T,), 1.0 / T, dtype=torch.float64) * (1 + 0.3 * torch.rand(T, dtype=torch.float64))
    return X, W, labels, rest, Gradients(X, W, labels, c, z, e), z, e


@pytest.mark.parametrize("T,H,V", [(6, 2048, 66536), (8, 520, 2100)])
def test_dx(T, H, V):
    X, W, labels, rest, G, z, e = _model(T, H, V, 1)
    right, bound = G.dX()
    labelled = set((labels // 64).tolist())
    for j in (0, V // 128, V // 64 - 1):           # any 64 rows of the vocabulary left out of D W
        if j in labelled:
            continue
        wrong = G.dX(skip=(64 * j, 64 * j + 64))[0]
        assert bool(((wrong - right).abs() > 2 * bound)[:, rest + j].all()), j
        twice = 2 * right - wrong
        assert bool(((twice - right).abs() > 2 * bound)[:, rest + j].all()), j
    assert _rejected(G.dX(skip=(0, V))[0], right, bound) > 0.3
    assert _rejected(G.dX(hot=0.0)[0], right, bound) > 0.01


def test_one_hot_part_of_dx_in_bf16():
    """The one-hot part's scale rounded to bf16, and then the sum stored in bf16: too far off; only stored: within the bound."""
    X, W, labels, rest, G, z, e = _model(64, 520, 2100, 4)
    right, bound = G.dX()
    stored = G.dX(c=G.c.to(torch.bfloat16).double())[0].to(torch.bfloat16).double()
    assert bool(((stored - right).abs() > bound).any())
    assert not bool(((right.to(torch.bfloat16).double() - right).abs() > bound).any())


def test_dw():
    T, H, V = 700, 256, 3000
    X, W, labels, rest, G, z, e = _model(T, H, V, 2)
    right, bound = G.dW()
    nv = -(-V // 64)
    unlabelled = torch.ones(V, dtype=torch.bool)
    unlabelled[labels] = False
    for b in (0, 5, T // 64):                      # any 64 tokens left out of D^T X
        wrong = G.dW(skip=(64 * b, 64 * b + 64))[0]
        assert bool(((wrong - right).abs() > 2 * bound)[unlabelled, rest + nv + b].all()), b
    assert _rejected(G.dW(skip=(0, T))[0], right, bound) > 0.02
    stored = G.dW(c=G.c.to(torch.bfloat16).double())[0].to(torch.bfloat16).double()
    assert bool(((stored - right).abs() > bound).any())
    assert not bool(((right.to(torch.bfloat16).double() - right).abs() > bound).any())


@pytest.mark.parametrize("kind", ["tc", "few", "fp32"])
def test_logits_rounded_to_bf16(kind):
    T, H, V = 8, 4096, 5001
    g = torch.Generator().manual_seed(3)
    X = torch.randn(T, H, generator=g).to(torch.bfloat16)
    W = (torch.randn(V, H, generator=g) * 1.3 * H ** -0.5).to(torch.bfloat16)
    labels = torch.randint(0, V, (T,), generator=g)
    z, e = logit_bounds(X, W, kind)
    lp, bound, *_ = logp_bounds(z, e, labels)
    cut = torch.log_softmax(z.to(torch.bfloat16).double(), 1).gather(1, labels[:, None])[:, 0]
    assert bool(((cut - lp).abs() > 2 * bound).any())
    assert float(bound.max()) < 2e-3
