"""References in 64 bits for the tests of the layer-norm layer's operators and of scored logits, from the formulas."""
import math

import torch

IGNORE = -100


def randn(gen, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def act(name, p):
    """The activation and its derivative, in p's precision."""
    if name == "none":
        return p, torch.ones_like(p)
    if name == "relu":
        return p.clamp(min=0), (p > 0).to(p.dtype)
    if name == "silu":
        s = torch.sigmoid(p)
        return p * s, s * (1 + p * (1 - s))
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-p / math.sqrt(2))
        return p * cdf, cdf + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (p + 0.044715 * p ** 3))
    return p * s, s + p * s * (1 - s) * c * (1 + 3 * 0.044715 * p * p)


def frequencies(R, theta, scaling="none", factor=1.0, low=1.0, high=32.0, orig_len=0.0, attn_factor=0.0):
    """Inverse frequencies and the factor on cos and sin, as liger_layer.h gives them."""
    if scaling == "ntk" and R > 2:
        theta = theta * factor ** (R / (R - 2))
    f = [theta ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "bands":
        c = [min(max((orig_len * v / (2 * math.pi) - low) / (high - low), 0), 1) for v in f]
        f = [v * (a + (1 - a) / factor) for v, a in zip(f, c)]
    if scaling == "yarn":
        d = [R * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
        lo, hi = max(math.floor(d[0]), 0), min(math.ceil(d[1]), R - 1)
        c = [min(max((i - lo) / max(hi - lo, 0.001), 0), 1) for i in range(R // 2)]
        f = [v * (1 - a + a / factor) for v, a in zip(f, c)]
    m = attn_factor or (0.1 * math.log(factor) + 1 if scaling == "yarn" and factor > 1 else 1.0)
    return torch.tensor(f, dtype=torch.float64, device="cuda"), m


def rotate(x, pos, f, m, R, pairing, sign=1.0):
    """x [B, S, H, D] in 64 bits, rotated by pos [B, S]; also the magnitudes of the terms."""
    phi = pos.double()[..., None, None] * f
    c, s = m * torch.cos(phi), sign * m * torch.sin(phi)
    out, mag = x.clone(), x.abs()
    ia = torch.arange(R // 2, device=x.device) * (2 if pairing == "interleaved" else 1)
    ib = ia + (1 if pairing == "interleaved" else R // 2)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = m * (a.abs() + b.abs())
    return out, mag


def scores(z, tokens, temp, k, ignore=IGNORE):
    """logp, row_max, log_sum, entropy, top_logp, top_ids of logits in 64 bits (rows with at least one number)."""
    z = z.double()
    m = z.max(1).values
    a = (z - m[:, None]) / temp
    ls = torch.logsumexp(a, 1)
    lp = a - ls[:, None]
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    ok = (tokens >= 0) & (tokens < z.shape[1])
    logp = lp.gather(1, torch.where(ok, tokens, 0)[:, None])[:, 0]
    logp = torch.where(tokens == ignore, torch.zeros_like(logp), torch.where(ok, logp, torch.full_like(logp, float("nan"))))
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    return logp, m, ls, ent, lp.gather(1, ids), ids
