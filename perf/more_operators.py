"""The operators of a decoder layer with layer norms and biased projections, and of scoring its logits, as they are measured.

Layer norm with its gradients, the projection with bias, activation and residual sum in its epilogue (with its gradients),
rotary positions on a part of each head with frequencies scaled for long contexts, and from the head's logits the
log-probabilities of given tokens with the entropy, the top alternatives and the gradient.

`own` selects what `run` computes: the plain forms in elementary torch operations, or this package's kernels.
Sizes are those of this repository's configurations (hidden 4096, intermediate 11008, 32 and 8 heads of 128, sequences of
8192 and 32768 tokens, vocabularies 128256 and 151936) and ragged ones between.
"""
import math
import random  # noqa: F401  (draw's argument is a random.Random)

import torch

own = False

BF16, F32 = "bf16", "f32"
IGNORE = -100
EPS = 1e-5


def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few sequences being decoded: the norm of one row each, where the latency of the call counts
        {"name": "norm_decode", "op": "norm", "rows": 4, "cols": 4096, "dtype": BF16, "bias": True, "grads": False,
         "residual": False},
        # a training sequence of 32768 tokens, forward and backward, the residual stream's gradient added to the norm's
        {"name": "norm_train", "op": "norm", "rows": 32768, "cols": 4096, "dtype": BF16, "bias": True, "grads": True,
         "residual": True},
        # fp32, rows that are no whole vectors
        {"name": "norm_ragged_f32", "op": "norm", "rows": 1324, "cols": 1001, "dtype": F32, "bias": True, "grads": True,
         "residual": False},
        # the MLP's first projection for a few sequences being decoded: the weight is read once
        {"name": "linear_decode", "op": "linear", "tokens": 4, "inputs": 4096, "outputs": 11008, "dtype": BF16,
         "act": "gelu_tanh", "bias": True, "residual": False, "grads": False},
        # the same of 8192 tokens, forward and backward of one training step
        {"name": "linear_train", "op": "linear", "tokens": 8192, "inputs": 4096, "outputs": 11008, "dtype": BF16,
         "act": "gelu_tanh", "bias": True, "residual": False, "grads": True},
        # a short ragged batch of a small model, the projection that ends in the residual stream
        {"name": "linear_ragged", "op": "linear", "tokens": 1111, "inputs": 1384, "outputs": 520, "dtype": BF16,
         "act": "none", "bias": True, "residual": True, "grads": True},
        # fp32 on odd sizes, as tests and small models have them
        {"name": "linear_odd_f32", "op": "linear", "tokens": 300, "inputs": 257, "outputs": 1001, "dtype": F32,
         "act": "gelu", "bias": True, "residual": True, "grads": True},
        # 32 query and 8 key heads of [4, 8192] tokens, half of each head rotated, frequencies scaled for a longer context:
        # the rotation out of the packed projections, and the backward's
        {"name": "rope_train", "op": "rope", "batch": 4, "seq": 8192, "q_heads": 32, "k_heads": 8, "head": 128, "rotary": 64,
         "dtype": BF16, "pairing": "half", "scaling": "yarn", "theta": 5e5, "far": False, "grads": True},
        # one token each of 24 sequences deep in their contexts, interleaved pairs of a quarter of each head
        {"name": "rope_decode_f32", "op": "rope", "batch": 24, "seq": 1, "q_heads": 32, "k_heads": 8, "head": 80, "rotary": 20,
         "dtype": F32, "pairing": "interleaved", "scaling": "bands", "theta": 1e4, "far": True, "grads": False},
        # one sampled token under a mask of allowed words: its log-probability and the 20 best alternatives
        {"name": "score_one_token", "op": "score", "tokens": 1, "vocab": 151936, "dtype": BF16, "top": 20,
         "temperature": 0.7, "masked": 0.5, "entropy": True, "grads": False},
        # a batch of answers scored, with 8 alternatives each
        {"name": "score_batch", "op": "score", "tokens": 4096, "vocab": 128256, "dtype": BF16, "top": 8,
         "temperature": 1.0, "masked": 0.0, "entropy": True, "grads": False},
        # a training step with an entropy bonus: forward, and the gradient of the logits; a vocabulary of odd size
        {"name": "score_train_f32", "op": "score", "tokens": 1500, "vocab": 32771, "dtype": F32, "top": 0,
         "temperature": 1.0, "masked": 0.0, "entropy": True, "grads": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "rope", "score", "score"])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "norm":
        cols = _log_int(rng, 32, 16384)
        if rng.random() < 0.6:
            cols = max(32, cols // 32 * 32)
        rows = _log_int(rng, 1, min(32768, 32768 * 4096 // cols // (2 if dtype == F32 else 1)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "bias": rng.random() < 0.8,
                "grads": rng.random() < 0.6, "residual": rng.random() < 0.5}
    if op == "linear":
        # (the mask of a relu jumps at 0, where the sums of the two sides differ in the last bit: it is not among these)
        case = {"op": op, "dtype": dtype, "act": rng.choice(["none", "gelu", "gelu_tanh", "silu"]),
                "bias": rng.random() < 0.8, "residual": rng.random() < 0.5, "grads": rng.random() < 0.6}
        if dtype == F32 or rng.random() < 0.15:     # fp32 and sizes of no whole vectors: small models and tests
            case.update(tokens=_log_int(rng, 1, 2048), inputs=_log_int(rng, 16, 2048), outputs=_log_int(rng, 16, 2048))
        else:
            case.update(tokens=_log_int(rng, 1, 8192), inputs=8 * _log_int(rng, 8, 512), outputs=8 * _log_int(rng, 8, 1376))
        return case
    if op == "rope":
        head = rng.choice([64, 80, 96, 128, 256])
        rotary = rng.choice([head, head // 2, head // 4])
        q_heads = rng.choice([8, 16, 32])
        decode = rng.random() < 0.4
        batch = _log_int(rng, 1, 128) if decode else rng.choice([1, 2, 4])
        seq = 1 if decode else _log_int(rng, 2, 32768 * 128 // head // batch)
        return {"op": op, "batch": batch, "seq": seq, "q_heads": q_heads, "k_heads": rng.choice([1, q_heads // 4, q_heads]),
                "head": head, "rotary": rotary, "dtype": dtype if seq * head * q_heads <= 1 << 24 else BF16,
                "pairing": rng.choice(["half", "half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "bands", "yarn"]), "theta": rng.choice([1e4, 5e5]),
                "far": decode, "grads": rng.random() < 0.5}
    vocab = _log_int(rng, 100, 151936)
    if rng.random() < 0.5:
        vocab = max(104, vocab // 8 * 8)
    tokens = _log_int(rng, 1, min(8192, 4096 * 128256 // 4 // vocab))
    return {"op": op, "tokens": tokens, "vocab": vocab, "dtype": dtype, "top": rng.choice([0, 1, 5, 8, 20]),
            "temperature": rng.choice([1.0, 1.0, round(rng.uniform(0.3, 2.0), 2)]), "masked": rng.choice([0.0, 0.0, 0.5, 0.9]),
            "entropy": rng.random() < 0.8, "grads": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------------ inputs
# Scaling of the frequencies: a model trained on orig_len positions and used on factor times as many.
ORIG_LEN, FACTOR = 8192, 8.0
BETA_SLOW, BETA_FAST = 1.0, 32.0        # yarn: rotations over orig_len
LOW, HIGH = 1.0, 4.0                    # bands: orig_len / wavelength


def _scaling(case):
    kind = case["scaling"]
    args = {"theta": case["theta"], "scaling": kind}
    if kind != "none":
        args["factor"] = FACTOR
    if kind in ("bands", "yarn"):
        args["orig_len"] = ORIG_LEN
        args["low"], args["high"] = (LOW, HIGH) if kind == "bands" else (BETA_SLOW, BETA_FAST)
    return args


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, op = _dt(case), case["op"]
    s = {"case": case}

    def randn(*shape, std=1.0, mean=0.0, dtype=None):
        return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(dtype or dt)

    if op == "norm":
        T, H = case["rows"], case["cols"]
        s["x"] = randn(T, H, std=1.5, mean=0.3)
        s["w"] = randn(H, std=0.1, mean=1.0)
        s["b"] = randn(H, std=0.1) if case["bias"] else None
        s["y"] = torch.empty_like(s["x"])
        s["mean"], s["rstd"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        if case["grads"]:
            s["dy"] = randn(T, H)
            s["dres"] = randn(T, H) if case["residual"] else None
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
            s["db"] = torch.empty_like(s["b"]) if case["bias"] else None
    elif op == "linear":
        T, H, N = case["tokens"], case["inputs"], case["outputs"]
        s["X"], s["W"] = randn(T, H), randn(N, H, std=1.28 / math.sqrt(H))
        s["bias"] = randn(N, std=0.3) if case["bias"] else None
        s["residual"] = randn(T, N, std=1.5) if case["residual"] else None
        s["Y"] = torch.empty(T, N, dtype=dt, device="cuda")
        # what the forward keeps for the activation's gradient: the sums before it, 16 bits an element (fp32: 32)
        s["pre"] = None
        if case["grads"] and case["act"] != "none":
            s["pre"] = torch.empty(T, N, dtype=torch.float16 if case["dtype"] == BF16 else dt, device="cuda")
        if case["grads"]:
            s["dY"] = randn(T, N)
            s["dX"], s["dW"] = torch.empty_like(s["X"]), torch.empty_like(s["W"])
            s["db"] = torch.empty_like(s["bias"]) if case["bias"] else None
    elif op == "rope":
        B, S, Hq, Hk, D = (case[k] for k in ("batch", "seq", "q_heads", "k_heads", "head"))
        packed = randn(B, S, Hq + 2 * Hk, D)        # the projections of q, k and v stand in one buffer
        s["q"], s["k"] = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hk]
        s["q_out"], s["k_out"] = (torch.empty(B, S, h, D, dtype=dt, device="cuda") for h in (Hq, Hk))
        s["pos"] = None
        if case["far"]:
            s["pos"] = torch.randint(0, int(ORIG_LEN * FACTOR), (B, S), device="cuda", generator=gen).to(torch.int32)
        if case["grads"]:
            for t, h in (("dq", Hq), ("dk", Hk)):
                s[t] = randn(B, S, h, D)
                s[t + "_out"] = torch.empty_like(s[t])
    else:
        T, V = case["tokens"], case["vocab"]
        z = torch.empty(T, V, dtype=dt, device="cuda")
        s["tokens"] = torch.empty(T, dtype=torch.int64, device="cuda")
        for t in range(0, T, 1024):
            part = z[t:t + 1024]
            part.copy_(torch.randn(part.shape, device="cuda", generator=gen) * 2.5)
            if case["masked"]:                      # words that a grammar or a filter has ruled out
                part.masked_fill_(torch.rand(part.shape, device="cuda", generator=gen) < case["masked"], float("-inf"))
                part[:, 0] = 1.0                    # the end of the answer is always allowed
            noise = torch.rand(part.shape, device="cuda", generator=gen).clamp_(1e-20, 1 - 1e-7)
            s["tokens"][t:t + 1024] = (part.float() / case["temperature"] - noise.log_().neg_().log_()).argmax(1)
        s["logits"] = z
        s["logp"], s["row_max"], s["log_sum"] = (torch.empty(T, device="cuda") for _ in range(3))
        s["entropy"] = torch.empty(T, device="cuda") if case["entropy"] else None
        k = min(case["top"], V)
        s["top_logp"] = torch.empty(T, k, device="cuda") if k else None
        s["top_ids"] = torch.empty(T, k, dtype=torch.int64, device="cuda") if k else None
        if case["grads"]:                           # a tenth of the tokens are prompts
            s["tokens"][torch.rand(T, device="cuda", generator=gen) < 0.1] = IGNORE
            s["g_logp"] = randn(T, dtype=torch.float32)
            s["g_entropy"] = randn(T, std=0.1, dtype=torch.float32) if case["entropy"] else None
            s["dlogits"] = torch.empty_like(z)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    return _OWN[op](s) if own else _PLAIN[op](s)


def _scratch(s, size):
    """The workspace that a program keeps from step to step."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(int(size()), 256), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_norm(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    L.liger_layernorm_fwd(s["x"], s["w"], s["b"], s["y"], mean=s["mean"], rstd=s["rstd"], eps=EPS)
    out = {k: s[k] for k in ("y", "mean", "rstd")}
    if c["grads"]:
        ws = _scratch(s, lambda: L.liger_layernorm_bwd_workspace(c["rows"], c["cols"]))
        L.liger_layernorm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"], ws, dres=s["dres"])
        out.update({k: s[k] for k in ("dx", "dw", "db")})
    return out


def _own_linear(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    L.liger_linear_act_fwd(s["X"], s["W"], s["Y"], bias=s["bias"], residual=s["residual"], act=c["act"], pre=s["pre"])
    out = {"Y": s["Y"]}
    if c["grads"]:
        ws = _scratch(s, lambda: L.liger_linear_act_bwd_workspace(c["tokens"], c["inputs"], c["outputs"], c["act"],
                                                                  L.LIGER_BF16 if c["dtype"] == BF16 else L.LIGER_F32))
        L.liger_linear_act_bwd(s["dY"], s["X"], s["W"], s["dX"], s["dW"], s["db"], ws, pre=s["pre"], act=c["act"])
        out.update({k: s[k] for k in ("dX", "dW", "db")})
    return out


def _own_rope(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    args = dict(pos=s["pos"], pairing=c["pairing"], **_scaling(c))
    L.liger_rope_scaled_fwd(s["q"], s["k"], s["q_out"], s["k_out"], c["rotary"], **args)
    out = {k: s[k] for k in ("q_out", "k_out")}
    if c["grads"]:
        L.liger_rope_scaled_bwd(s["dq"], s["dk"], s["dq_out"], s["dk_out"], c["rotary"], **args)
        out.update({k: s[k] for k in ("dq_out", "dk_out")})
    return out


def _own_score(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    L.liger_token_logp_fwd(s["logits"], s["tokens"], s["logp"], row_max=s["row_max"], log_sum=s["log_sum"],
                           entropy=s["entropy"], top_logp=s["top_logp"], top_ids=s["top_ids"],
                           temperature=c["temperature"], ignore_index=IGNORE)
    out = {k: s[k] for k in ("logp", "row_max", "log_sum", "entropy", "top_logp", "top_ids")}
    if c["grads"]:
        L.liger_token_logp_bwd(s["logits"], s["tokens"], s["row_max"], s["log_sum"], s["g_logp"], s["dlogits"],
                               entropy=s["entropy"], g_entropy=s["g_entropy"], temperature=c["temperature"],
                               ignore_index=IGNORE)
        out["dlogits"] = s["dlogits"]
    return out


_OWN = {"norm": _own_norm, "linear": _own_linear, "rope": _own_rope, "score": _own_score}


# ------------------------------------------------------------------------------------------------ plain forms (32 bits)
def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + EPS)
    xh = xc * rstd[:, None]
    y = xh * w
    if c["bias"]:
        y = y + s["b"].float()
    out = {"y": y.to(dt), "mean": mean, "rstd": rstd}
    if c["grads"]:
        dy = s["dy"].float()
        g = dy * w
        dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dres"].float()
        out.update(dx=dx.to(dt), dw=(dy * xh).sum(0).to(dt), db=dy.sum(0).to(dt) if c["bias"] else None)
    return out


ROOT_2_PI = math.sqrt(2.0 / math.pi)


def _plain_act(act, p):
    """The activation of p and its derivative."""
    if act == "none":
        return p, torch.ones_like(p)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-p))
        return p * sig, sig * (1.0 + p * (1.0 - sig))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(p * math.sqrt(0.5)))
        return p * cdf, cdf + p * torch.exp(-0.5 * p * p) * (1.0 / math.sqrt(2.0 * math.pi))
    t = torch.tanh(ROOT_2_PI * (p + 0.044715 * p * p * p))
    return 0.5 * p * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * ROOT_2_PI * (1.0 + 3 * 0.044715 * p * p)


def _plain_linear(s):
    c, dt = s["case"], s["X"].dtype
    X, W = s["X"].float(), s["W"].float()
    p = X @ W.T
    if c["bias"]:
        p = p + s["bias"].float()
    y, slope = _plain_act(c["act"], p)
    if c["residual"]:
        y = y + s["residual"].float()
    out = {"Y": y.to(dt)}
    if c["grads"]:
        dp = s["dY"].float() * slope
        out.update(dX=(dp @ W).to(dt), dW=(dp.T @ X).to(dt), db=dp.sum(0).to(dt) if c["bias"] else None)
    return out


def _frequencies(case, device):
    """Inverse frequencies (64 bits) of the rotated pairs, and the factor on cos and sin."""
    R, theta, kind = case["rotary"], case["theta"], case["scaling"]
    i = torch.arange(R // 2, dtype=torch.float64, device=device)
    if kind == "ntk" and R > 2:
        theta = theta * FACTOR ** (R / (R - 2))
    f = theta ** (-2.0 * i / R)
    if kind == "linear":
        f = f / FACTOR
    if kind == "bands":
        turns = ORIG_LEN * f / (2 * math.pi)        # orig_len / wavelength
        blend = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * (blend + (1 - blend) / FACTOR)
    if kind == "yarn":
        def dim(rotations):
            return R * math.log(ORIG_LEN / (rotations * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(BETA_FAST)), 0), min(math.ceil(dim(BETA_SLOW)), R - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / FACTOR * ramp
    return f, 0.1 * math.log(FACTOR) + 1.0 if kind == "yarn" else 1.0


def _plain_rope(s):
    c = s["case"]
    B, S, R = c["batch"], c["seq"], c["rotary"]
    f, m = _frequencies(c, s["q"].device)
    p = s["pos"] if s["pos"] is not None else torch.arange(S, device=f.device)[None].expand(B, S)
    phi = p.double()[..., None] * f
    cos, sin = ((m * g(phi)).float()[:, :, None] for g in (torch.cos, torch.sin))

    def rotate(x, sin):
        out = x.float()
        a, b = (out[..., 0:R:2], out[..., 1:R:2]) if c["pairing"] == "interleaved" else (out[..., :R // 2], out[..., R // 2:R])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((ra, rb), -1).flatten(-2) if c["pairing"] == "interleaved" else torch.cat((ra, rb), -1)
        return torch.cat((turned.to(x.dtype), x[..., R:]), -1)

    out = {"q_out": rotate(s["q"], sin), "k_out": rotate(s["k"], sin)}
    if c["grads"]:
        out.update(dq_out=rotate(s["dq"], -sin), dk_out=rotate(s["dk"], -sin))
    return out


def _plain_score(s):
    c, tokens = s["case"], s["tokens"]
    T, V = c["tokens"], c["vocab"]
    k = min(c["top"], V)
    logp, top, log_sum, ent = (torch.empty(T, device="cuda") for _ in range(4))
    top_logp = torch.empty(T, k, device="cuda")
    top_ids = torch.empty(T, k, dtype=torch.int64, device="cuda")
    dz = torch.empty_like(s["logits"]) if c["grads"] else None
    for t in range(0, T, 512):
        at = slice(t, t + 512)
        z = s["logits"][at].float()
        if k:                                       # ties: the lowest index first
            best, ids = torch.sort(z, dim=1, descending=True, stable=True)
            best, top_ids[at] = best[:, :k] / c["temperature"], ids[:, :k]
            del ids
        top[at] = z.amax(1)
        z = z / c["temperature"]
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        p = e / total
        log_sum[at] = total.log()[:, 0]
        lp = z - m - total.log()
        y = tokens[at]
        live = y != IGNORE
        logp[at] = torch.where(live, lp.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
        if k:
            top_logp[at] = best - m - total.log()
        lp = torch.where(p > 0, lp, 0.0)
        h = -(p * lp).sum(1, keepdim=True)
        ent[at] = h[:, 0]
        if c["grads"]:
            g = torch.where(live, s["g_logp"][at], 0.0)[:, None]
            d = -g * p
            if c["entropy"]:
                d = d - s["g_entropy"][at][:, None] * p * (lp + h)
            d.scatter_add_(1, y.clamp(min=0)[:, None], g)
            dz[at] = (d / c["temperature"]).to(dz.dtype)
    out = {"logp": logp, "row_max": top, "log_sum": log_sum, "entropy": ent if c["entropy"] else None,
           "top_logp": top_logp if k else None, "top_ids": top_ids if k else None}
    if c["grads"]:
        out["dlogits"] = dz
    return out


_PLAIN = {"norm": _plain_norm, "linear": _plain_linear, "rope": _plain_rope, "score": _plain_score}


# ------------------------------------------------------------------------------------------------ least work
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == BF16 else 4
    if op == "norm":
        T, n, H = case["rows"], case["rows"] * case["cols"], case["cols"]
        vectors = H * (1 + case["bias"])
        w = {"bytes": e * (2 * n + vectors) + 8 * T, "flops": 8.0 * n}
        if case["grads"]:       # x, dy (and dres) in, dx out, the weight in, its gradients out
            w["bytes"] += e * (n * (3 + case["residual"]) + H + vectors) + 8 * T
            w["flops"] += 16.0 * n
        return w
    if op == "linear":
        T, H, N = case["tokens"], case["inputs"], case["outputs"]
        kept = T * N if case["grads"] and case["act"] != "none" else 0
        w = {"bytes": e * (T * H + N * H + T * N * (1 + case["residual"]) + N * case["bias"] + kept), "flops": 2.0 * T * H * N}
        if case["grads"]:       # dY, X, W and what was kept in, dX, dW and the bias' gradient out
            w["bytes"] += e * (T * N + 2 * T * H + 2 * N * H + kept + N * case["bias"])
            w["flops"] += 4.0 * T * H * N
        return w
    if op == "rope":
        n = case["batch"] * case["seq"] * (case["q_heads"] + case["k_heads"])
        passes = 1 + case["grads"]
        return {"bytes": passes * (2 * e * n * case["head"] + 4 * case["batch"] * case["seq"] * case["far"]),
                "flops": passes * 3.0 * n * case["rotary"]}
    T, V, k = case["tokens"], case["vocab"], case["top"]
    w = {"bytes": e * T * V + T * (20 + 4 * case["entropy"] + 12 * k), "flops": 6.0 * T * V}
    if case["grads"]:
        w["bytes"] += 2 * e * T * V + T * (20 + 8 * case["entropy"])
        w["flops"] += 8.0 * T * V
    return w


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, {k: v.double() if torch.is_tensor(v) and v.is_floating_point() and case["op"] != "score"
                                     else v for k, v in s.items()})


def _exact_norm(c, d):
    x, H = d["x"], c["cols"]
    mean = x.sum(1) / H
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / H + EPS)
    y = torch.einsum("th,t,h->th", x - mean[:, None], rstd, d["w"])
    out = {"y": y + d["b"] if c["bias"] else y, "mean": mean, "rstd": rstd}
    if c["grads"]:
        xc = x - mean[:, None]
        u = d["dy"] * d["w"]
        s1, s2 = u.sum(1) / H, (u * xc).sum(1) / H
        dx = (u - s1[:, None]) * rstd[:, None] - xc * (rstd ** 3 * s2)[:, None]
        out["dx"] = dx + d["dres"] if c["residual"] else dx
        out["dw"] = torch.einsum("th,th,t->h", d["dy"], xc, rstd)
        out["db"] = d["dy"].sum(0) if c["bias"] else None
    return out


def _exact_linear(c, d):
    p = torch.nn.functional.pad(d["X"], (0, 1), value=1.0) @ torch.cat(
        (d["W"], (d["bias"] if c["bias"] else torch.zeros_like(d["W"][:, 0]))[:, None]), 1).T
    if c["act"] == "none":
        y, slope = p, torch.ones_like(p)
    elif c["act"] == "silu":
        y = p * torch.sigmoid(p)
        slope = torch.sigmoid(p) + y * torch.sigmoid(-p)
    elif c["act"] == "gelu":
        y = p * torch.special.ndtr(p)
        slope = torch.special.ndtr(p) + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    else:       # p (1 + tanh a) / 2 = p sigmoid(2 a)
        a = 2 * ROOT_2_PI * (p + 0.044715 * p ** 3)
        y = p * torch.sigmoid(a)
        slope = torch.sigmoid(a) + y * torch.sigmoid(-a) * 2 * ROOT_2_PI * (1 + 0.134145 * p ** 2)
    out = {"Y": y + d["residual"] if c["residual"] else y}
    if c["grads"]:
        dp = d["dY"] * slope
        out.update(dX=dp @ d["W"], dW=dp.T @ d["X"], db=dp.sum(0) if c["bias"] else None)
    return out


def _exact_rope(c, d):
    S, R = c["seq"], c["rotary"]
    step = [c["theta"] ** (-2.0 * i / R) for i in range(R // 2)]
    grow = 1.0
    if c["scaling"] == "linear":
        step = [f / FACTOR for f in step]
    elif c["scaling"] == "ntk" and R > 2:
        step = [f * FACTOR ** (-2.0 * i / (R - 2)) for i, f in enumerate(step)]
    elif c["scaling"] == "bands":
        for i, f in enumerate(step):
            wave = 2 * math.pi / f
            if wave > ORIG_LEN / LOW:
                step[i] = f / FACTOR
            elif wave > ORIG_LEN / HIGH:
                w = (ORIG_LEN / wave - LOW) / (HIGH - LOW)
                step[i] = (1 - w) * f / FACTOR + w * f
    elif c["scaling"] == "yarn":
        ends = [R / 2 * math.log(ORIG_LEN / (2 * math.pi * b), c["theta"]) for b in (BETA_FAST, BETA_SLOW)]
        lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), R - 1)
        for i, f in enumerate(step):
            w = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            step[i] = f * ((1 - w) + w / FACTOR)
        grow = 1.0 + math.log(FACTOR) / 10
    step = torch.tensor(step, dtype=torch.float64, device="cuda")
    pos = torch.arange(S, device="cuda")[None] if d["pos"] is None else d["pos"]
    turn = torch.polar(torch.full_like(step, grow), torch.zeros_like(step)) * torch.exp(1j * (pos.double()[..., None] * step))

    def rotate(x, turn):
        head = x[..., :R].contiguous()
        pairs = head.unflatten(-1, (R // 2, 2)) if c["pairing"] == "interleaved" else \
            head.unflatten(-1, (2, R // 2)).transpose(-1, -2).contiguous()
        z = torch.view_as_real(torch.view_as_complex(pairs) * turn[:, :, None])
        z = z.flatten(-2) if c["pairing"] == "interleaved" else z.transpose(-1, -2).flatten(-2)
        return torch.cat((z, x[..., R:]), -1)

    out = {"q_out": rotate(d["q"], turn), "k_out": rotate(d["k"], turn)}
    if c["grads"]:
        out.update(dq_out=rotate(d["dq"], turn.conj()), dk_out=rotate(d["dk"], turn.conj()))
    return out


def _exact_score(c, d):
    T, k = c["tokens"], min(c["top"], c["vocab"])
    parts = {"logp": [], "row_max": [], "log_sum": [], "entropy": [], "top_logp": [], "top_ids": [], "dlogits": []}
    for t in range(0, T, 256):
        at = slice(t, t + 256)
        z = d["logits"][at].double() / c["temperature"]
        lse = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        ent = torch.special.entr(p).sum(1)
        y, rows = d["tokens"][at], torch.arange(z.shape[0], device=z.device)
        live = y >= 0
        parts["logp"].append(torch.where(live, z[rows, y.clamp(min=0)] - lse, 0.0))
        parts["row_max"].append(d["logits"][at].double().max(1).values)
        parts["log_sum"].append(torch.logsumexp(z - z.max(1, keepdim=True).values, 1))
        parts["entropy"].append(ent)
        if k:
            ids = torch.argsort(z, dim=1, descending=True, stable=True)[:, :k]
            parts["top_ids"].append(ids)
            parts["top_logp"].append(z.gather(1, ids) - lse[:, None])
        if c["grads"]:
            hot = torch.zeros_like(p)
            hot[rows[live], y[live]] = 1.0
            dz = (hot - p) * torch.where(live, d["g_logp"][at].double(), 0.0)[:, None]
            if c["entropy"]:
                dz = dz + d["g_entropy"][at].double()[:, None] * (torch.special.entr(p) - p * ent[:, None])
            parts["dlogits"].append(dz / c["temperature"])
    out = {n: torch.cat(v) if v else None for n, v in parts.items()}
    if not c["entropy"]:
        out["entropy"] = None
    if not c["grads"]:
        del out["dlogits"]
    return out


_EXACT = {"norm": _exact_norm, "linear": _exact_linear, "rope": _exact_rope, "score": _exact_score}
