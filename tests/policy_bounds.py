"""Inputs and bounds of the policy loss and the log-probabilities under which a missing part shows.

The inputs carry signatures.  Column 64-block j of the vocabulary has a hidden column of its own, where W is between 1 and 2
for the block's rows and 0 elsewhere and X is 0: dX there is c (P(block) W - W[y]) of that block alone, a sum of one sign, so a
k range of dX = D W that is left out, doubled or misplaced changes a column by its whole value.  Likewise every 64 tokens have a
column where X is between 1 and 2 for them and W is 0, for dW = D^T X.  The remaining columns make the logits.

The bounds, from the arithmetic (u = 2^-8 the half step of bf16):
  * a logit: the tensor cores add 16 exact products and the running sum, each of the 17 cut off at the last place of the
    largest: 17 2^-23 (|sum so far| + sum |products of the step|) a step, over the steps.  Off the tensor cores fp32 fma:
    16 2^-24 of the same for 16 of them, and of the sum where a run of K starts, at most the largest.  The few-token kernel: a
    lane adds H / 64 products in each of two sums, 6 more adds: (H / 64 + 8) 2^-24 sum |products|;
  * a log-probability: the label's logit, the softmax-weighted mean of the logits' bounds, and 2^-20 (the exponentials' 2^-21
    and their sum) + 2^-22 (|z| + |lse|);
  * c = r A w: the change of lp, and 2^-20 for exp and the products;
  * a softmax weight c p in D: P and D rounded to bf16, 2 u + u^2; the logit's, lse's and c's bounds; 2^-20 (4 + |z| + |lse|) for
    the exponents' arguments.  Its sum: 17 2^-23 of the terms' sizes for each step of 16 that is not all zeros;
  * the one-hot part: c's bound and 2^-22, no rounding to bf16;
  * the stored gradient: u of its value."""
import torch

U = 2.0 ** -8


def signed_inputs(T, H, V, seed, device, masked=0.0, dtype=torch.bfloat16):
    g = torch.Generator(device=device).manual_seed(seed)
    nv, nt = -(-V // 64), -(-T // 64)
    rest = H - nv - nt
    assert rest >= 64
    X = torch.randn(T, H, device=device, generator=g)
    W = torch.randn(V, H, device=device, generator=g) * (1.3 * rest ** -0.5)
    X[:, rest:] = 0
    W[:, rest:] = 0
    v, t = torch.arange(V, device=device), torch.arange(T, device=device)
    W[v, rest + v // 64] = 1 + torch.rand(V, device=device, generator=g)
    X[t, rest + nv + t // 64] = 1 + torch.rand(T, device=device, generator=g)
    labels = torch.randint(0, V, (T,), device=device, generator=g)
    labels[torch.rand(T, device=device, generator=g) < masked] = -100
    return X.to(dtype), W.to(dtype), labels, rest


def logit_bounds(X, W, kind):
    """z and its bound for all tokens and rows, in 64 bits; kind: tc, few, fp32."""
    x, H = X.double(), X.shape[1]
    z = torch.empty(X.shape[0], W.shape[0], dtype=torch.float64, device=X.device)
    e = torch.empty_like(z)
    for a in range(0, W.shape[0], 8192):
        w = W[a:a + 8192].double()
        size = x.abs() @ w.abs().T
        if kind == "few":
            z[:, a:a + 8192] = x @ w.T
            e[:, a:a + 8192] = (H / 64 + 8) * 2.0 ** -24 * size
            continue
        s, run, top = torch.zeros_like(size), torch.zeros_like(size), torch.zeros_like(size)
        for k in range(0, H, 16):
            run += s.abs()
            s = s + x[:, k:k + 16] @ w[:, k:k + 16].T
            if kind == "fp32":
                top = torch.maximum(top, s.abs())
        z[:, a:a + 8192] = s
        if kind == "tc":
            e[:, a:a + 8192] = 17 * 2.0 ** -23 * (run + s.abs() + size)
        else:
            e[:, a:a + 8192] = 16 * 2.0 ** -24 * (run + s.abs() + size + (H / 16 + 2) * top)
    return z, e


def logp_bounds(z, e, labels):
    """lp of tokens that all have a label, its bound, lse and its bound, softmax."""
    at = labels[:, None]
    zy, lse = z.gather(1, at)[:, 0], torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    e_lse = (p * e).sum(1) + 2.0 ** -20 + 2.0 ** -22 * lse.abs()
    return zy - lse, e.gather(1, at)[:, 0] + e_lse + 2.0 ** -22 * zy.abs(), lse, e_lse, p


class Gradients:
    """dX and dW of tokens with scales c (all have a label), and how far the kernels may be off; bf16 tensor-core path."""

    def __init__(self, X, W, labels, c, z, e, spread=1.0):
        self.spread = spread        # tokens among the rows of the GEMMs for each that has a label
        self.x, self.W, self.labels, self.c = X.double(), W, labels, c
        self.lp, self.e_lp, lse, e_lse, self.p = logp_bounds(z, e, labels)
        self.e_c = self.e_lp + 2.0 ** -20
        rel = 2 * U + U * U + e + (e_lse + self.e_c)[:, None] + 2.0 ** -20 * (4 + z.abs() + lse.abs()[:, None])
        self.soft = self.p * c[:, None]
        self.off = self.soft.abs() * rel

    def dX(self, rows=slice(None), skip=None, hot=1.0, c=None):
        """Rows of dX and their bound; skip: vocabulary range left out of D W; hot: factor of the one-hot part; c: its scale."""
        soft, off, y = self.soft[rows], self.off[rows], self.labels[rows]
        out, bound, steps = 0.0, 0.0, 0.0
        for a in range(0, self.W.shape[0], 8192):
            w = self.W[a:a + 8192].double()
            keep = soft[:, a:a + 8192]
            if skip is not None:
                v = torch.arange(a, a + w.shape[0], device=w.device)
                keep = keep * ~((v >= skip[0]) & (v < skip[1]))
            out = out + keep @ w
            bound = bound + off[:, a:a + 8192] @ w.abs()
            n = torch.nn.functional.pad(w, (0, 0, 0, -w.shape[0] % 16)).view(-1, 16, w.shape[1])
            steps = steps + (n != 0).any(1).sum(0)
        size = torch.zeros_like(out)
        for a in range(0, self.W.shape[0], 8192):
            size += soft[:, a:a + 8192].abs() @ self.W[a:a + 8192].double().abs()
        one = (self.c[rows] if c is None else c[rows])[:, None] * self.W[y].double()
        bound = bound + 17 * 2.0 ** -23 * (steps + 1) * size + (self.e_c[rows][:, None] + 2.0 ** -22) * one.abs()
        out = out - hot * one
        return out, (1 + U) * bound + U * out.abs()

    def dW(self, rows=slice(None), skip=None, hot=1.0, c=None):
        """Rows of dW and their bound; skip: range of tokens left out of D^T X."""
        soft, off = self.soft[:, rows], self.off[:, rows]
        keep = soft
        if skip is not None:
            t = torch.arange(soft.shape[0], device=soft.device)
            keep = soft * ~((t >= skip[0]) & (t < skip[1]))[:, None]
        size = soft.abs().T @ self.x.abs()
        pad = torch.nn.functional.pad(self.x, (0, 0, 0, -self.x.shape[0] % 16)).view(-1, 16, self.x.shape[1])
        steps = (pad != 0).any(1).sum(0) * self.spread + 2
        v = torch.arange(self.W.shape[0], device=soft.device)[rows]
        one = (self.labels[:, None] == v).double()
        cc = self.c if c is None else c
        hots = one.T @ (cc[:, None] * self.x)
        hot_off = one.T @ ((self.c.abs() * self.e_c)[:, None] * self.x.abs())
        hot_size = one.T @ (self.c.abs()[:, None] * self.x.abs())
        n = one.sum(0)[:, None]
        out = keep.T @ self.x - hot * hots
        bound = off.T @ self.x.abs() + 17 * 2.0 ** -23 * steps * size + hot_off + (2.0 ** -22 + n * 2.0 ** -24) * hot_size
        return out, (1 + U) * bound + U * out.abs()
