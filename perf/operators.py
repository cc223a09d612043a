"""The operators of a policy-optimisation step of a decoder, as they are measured.

Block norms (the norm behind a block, its gate, the scaled residual sum and the norm before the next block), SwiGLU whose
gate and up values are kept for the backward in 8 bits (alone, and inside the fused gate/up projections), the label
log-probabilities of a linear head, and the clipped policy loss with a KL term from the hidden states, with its gradients.

`own` selects what `run` computes: the plain forms in elementary torch operations, or this package's kernels.
Sizes are those of this repository's configurations (hidden 4096 and 256, intermediate 11008, vocabularies 128256, 151936
and 1024) and ragged ones between.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
GROUP = 32      # columns of a row that share one step in an 8-bit checkpoint
IGNORE = -100
EPS = 1e-6


def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few sequences being decoded: one row each, where the latency of the call counts
        {"name": "norms_fwd_decode", "op": "norms_fwd", "rows": 4, "cols": 4096, "dtype": BF16, "post": True, "pre": True,
         "gates": 0, "res_scale": 1.0, "block_scale": 1.0, "grad_h": False},
        # a training sequence of 32768 tokens with a learned gate for each channel
        {"name": "norms_fwd_train", "op": "norms_fwd", "rows": 32768, "cols": 4096, "dtype": BF16, "post": True, "pre": True,
         "gates": 1, "res_scale": 1.0, "block_scale": 1.0, "grad_h": False},
        # its backward: the gradients of both streams, of both norm weights and of the gate
        {"name": "norms_bwd_train", "op": "norms_bwd", "rows": 32768, "cols": 4096, "dtype": BF16, "post": True, "pre": True,
         "gates": 1, "res_scale": 1.0, "block_scale": 1.0, "grad_h": True},
        # fp32, rows that are no whole vectors, one gate for each of four sequences, scaled residual
        {"name": "norms_bwd_ragged_f32", "op": "norms_bwd", "rows": 1324, "cols": 1001, "dtype": F32, "post": True,
         "pre": True, "gates": 4, "res_scale": 0.75, "block_scale": 0.5, "grad_h": True},
        # the activation of [4, 2048, 11008], forward and backward of one training step
        {"name": "swiglu8_train", "op": "swiglu8", "rows": 8192, "cols": 11008, "dtype": BF16},
        # fp32 rows that end inside a checkpoint group
        {"name": "swiglu8_ragged_f32", "op": "swiglu8", "rows": 515, "cols": 2739, "dtype": F32},
        # the MLP's projections of 8192 tokens, forward and backward of one training step
        {"name": "linear_swiglu8_train", "op": "linear_swiglu8", "tokens": 8192, "hidden": 4096, "inter": 11008, "dtype": BF16},
        # a short ragged batch of a small model
        {"name": "linear_swiglu8_ragged", "op": "linear_swiglu8", "tokens": 1111, "hidden": 520, "inter": 1384, "dtype": BF16},
        # a policy step on eight answers with masked prompts at a 128256-word head
        {"name": "policy_train", "op": "policy", "tokens": 4096, "hidden": 4096, "vocab": 128256, "dtype": BF16, "seqs": 8,
         "reduction": "seq_mean", "beta": 0.04, "eps_low": 0.2, "eps_high": 0.2},
        # the same in fp32 on the tiny configuration
        {"name": "policy_tiny_f32", "op": "policy", "tokens": 256, "hidden": 256, "vocab": 1024, "dtype": F32, "seqs": 5,
         "reduction": "token_mean", "beta": 0.1, "eps_low": 0.2, "eps_high": 0.28},
        # the reference policy's log-probabilities of a batch
        {"name": "logp_batch", "op": "logp", "tokens": 8192, "hidden": 4096, "vocab": 151936, "dtype": BF16, "seqs": 8},
        # one token scored: the head's weight is read once
        {"name": "logp_one_token", "op": "logp", "tokens": 1, "hidden": 4096, "vocab": 128256, "dtype": BF16, "seqs": 1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norms_fwd", "norms_bwd", "swiglu8", "linear_swiglu8", "policy", "logp"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("norms_fwd", "norms_bwd"):
        cols = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, min(32768, 32768 * 4096 // cols // (2 if dtype == F32 else 1)))
        gates = rng.choice([0, 1, 1, 2])
        if gates == 2:      # a gate for each of several sequences of one length
            gates = _log_int(rng, 1, rows)
            rows = rows // gates * gates
        post = rng.random() < 0.8
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "post": post, "pre": not post or rng.random() < 0.85,
                "gates": gates, "res_scale": rng.choice([1.0, round(rng.uniform(0.2, 1.5), 3)]),
                "block_scale": rng.choice([1.0, round(rng.uniform(0.1, 1.5), 3)]), "grad_h": rng.random() < 0.85}
    if op == "swiglu8":
        cols = _log_int(rng, 16, 16384)
        if rng.random() < 0.5:
            cols = cols // 16 * 16
        rows = _log_int(rng, 1, min(32768, 8192 * 11008 // cols // (2 if dtype == F32 else 1)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype}
    if op == "linear_swiglu8":
        hidden, inter = 8 * _log_int(rng, 8, 512), 8 * _log_int(rng, 1, 1376)
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "hidden": hidden, "inter": inter, "dtype": BF16}
    if dtype == F32:        # fp32 heads are those of small models and of tests
        tokens, hidden, vocab = _log_int(rng, 1, 512), _log_int(rng, 32, 512), _log_int(rng, 16, 4096)
    else:
        tokens, hidden, vocab = _log_int(rng, 1, 4096), 8 * _log_int(rng, 8, 512), _log_int(rng, 256, 151936)
        if tokens * hidden * vocab > 4096 * 4096 * 128256:
            vocab = 4096 * 4096 * 128256 // (tokens * hidden)
    seqs = _log_int(rng, 1, min(tokens, 32))
    case = {"op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab, "dtype": dtype, "seqs": seqs}
    if op == "policy":
        case.update(reduction=rng.choice(["token_mean", "seq_mean", "sum"]), beta=rng.choice([0.0, 0.04, 0.1]),
                    eps_low=0.2, eps_high=rng.choice([0.2, 0.28]))
    return case


# ------------------------------------------------------------------------------------------------ inputs
def _layout(case):
    """Sequence starts and masked tokens of a packed batch: prompts are masked, now and then a whole answer; tokens may
    stand behind the last sequence (padding). From the case alone, so that the work is known without the inputs."""
    T, B = case["tokens"], case["seqs"]
    rng = random.Random(T * 1000003 + B)
    end = T if T < 64 or rng.random() < 0.5 else T - rng.randint(1, T // 32)
    cuts = sorted(rng.sample(range(1, end), B - 1)) if B > 1 else []
    starts = [0] + cuts + [end]
    valid = [False] * T
    for b in range(B):
        s, e = starts[b], starts[b + 1]
        if e - s > 1 and B > 4 and b == B // 2:
            continue                                    # an answer that was thrown out
        first = s + int((e - s) * rng.uniform(0.05, 0.4)) if e - s > 2 else s
        for t in range(first, e):
            valid[t] = True
    return starts, valid


def _head_inputs(case, gen):
    """Hidden states and head of the configurations' distributions, labels drawn from the model's own softmax, and (for a
    policy step) their log-probabilities."""
    T, H, V, dt = case["tokens"], case["hidden"], case["vocab"], _dt(case)
    X = torch.randn(T, H, device="cuda", generator=gen).to(dt)
    W = (torch.randn(V, H, device="cuda", generator=gen) * (1.28 / math.sqrt(H))).to(dt)
    labels = torch.empty(T, dtype=torch.int64, device="cuda")
    lp = torch.empty(T, device="cuda")
    for t in range(0, T, 1024):
        z = (X[t:t + 1024].bfloat16() @ W.bfloat16().T).float()
        noise = torch.rand(z.shape, device="cuda", generator=gen).clamp_(1e-20, 1 - 1e-7)
        y = (z - noise.log_().neg_().log_()).argmax(1)
        labels[t:t + 1024] = y
        if case["op"] == "policy":
            z = X[t:t + 1024].float() @ W.float().T
            lp[t:t + 1024] = (z.gather(1, y[:, None])[:, 0] - torch.logsumexp(z, 1))
    starts, valid = _layout(case)
    valid = torch.tensor(valid, device="cuda")
    labels[~valid] = IGNORE
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return X, W, labels, lp, valid, cu


def _log_ratio(case, d):
    """Log ratios of the new policy to the old, none of them at the edge of the clip range, where the gradient jumps."""
    for edge in (math.log(1 - case["eps_low"]), math.log(1 + case["eps_high"])):
        d = torch.where((d - edge).abs() < 1e-3, edge + 2e-3, d)
    return d


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, op = _dt(case), case["op"]
    s = {"case": case}

    def randn(*shape, std=1.0, mean=0.0, dtype=None):
        return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(dtype or dt)

    if op in ("norms_fwd", "norms_bwd"):
        T, H, G = case["rows"], case["cols"], case["gates"]
        s["z"] = randn(T, H)
        s["w_post"] = randn(H, std=0.1, mean=1.0) if case["post"] else None
        s["w_pre"] = randn(H, std=0.1, mean=1.0) if case["pre"] else None
        s["gate"] = randn(G, H, std=0.3, mean=0.5) if G else None
        if op == "norms_fwd":
            s["r"] = randn(T, H, std=1.5)
            s["h"] = torch.empty_like(s["z"])
            s["y"] = torch.empty_like(s["z"]) if case["pre"] else None
        else:
            s["h"] = randn(T, H, std=1.5)
            s["dy"] = randn(T, H) if case["pre"] else None
            s["dh"] = randn(T, H) if case["grad_h"] or not case["pre"] else None
            s["dr"], s["dz"] = torch.empty_like(s["z"]), torch.empty_like(s["z"])
            for k, v in (("dw_post", "w_post"), ("dgate", "gate"), ("dw_pre", "w_pre")):
                s[k] = torch.empty_like(s[v]) if s[v] is not None else None
        if op == "norms_fwd":
            s["rstd_z"] = torch.empty(T, device="cuda") if case["post"] else None
            s["rstd_h"] = torch.empty(T, device="cuda") if case["pre"] else None
        else:       # as the forward left them
            s["rstd_z"] = (s["z"].double().square().mean(1) + EPS).rsqrt().float() if case["post"] else None
            s["rstd_h"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float() if case["pre"] else None
    elif op == "swiglu8":
        T, I = case["rows"], case["cols"]
        s["gate"], s["up"], s["dy"] = randn(T, I), randn(T, I), randn(T, I)
        for k in ("y", "dgate", "dup"):
            s[k] = torch.empty_like(s["gate"])
        _checkpoints(s, T, I)
    elif op == "linear_swiglu8":
        T, H, I = case["tokens"], case["hidden"], case["inter"]
        s["X"], s["dH"] = randn(T, H), randn(T, I)
        s["Wg"], s["Wu"] = randn(I, H, std=1.28 / math.sqrt(H)), randn(I, H, std=1.28 / math.sqrt(H))
        s["out"], s["dX"] = torch.empty_like(s["dH"]), torch.empty_like(s["X"])
        s["dWg"], s["dWu"] = torch.empty_like(s["Wg"]), torch.empty_like(s["Wu"])
        _checkpoints(s, T, I)
    else:
        T, B = case["tokens"], case["seqs"]
        s["X"], s["W"], s["labels"], lp, valid, s["cu"] = _head_inputs(case, gen)
        s["logp"] = torch.empty(T, device="cuda")
        if op == "policy":
            nan = torch.full_like(lp, float("nan"))     # what stands in masked places is not read
            s["old"] = torch.where(valid, lp - _log_ratio(case, randn(T, std=0.2, dtype=torch.float32)), nan)
            s["ref"] = torch.where(valid, lp + randn(T, std=0.4, dtype=torch.float32), nan) if case["beta"] else None
            s["adv"] = randn(B, dtype=torch.float32)
            s["loss"], s["stats"] = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
            s["dX"], s["dW"] = torch.empty_like(s["X"]), torch.empty_like(s["W"])
    return s


def _checkpoints(s, rows, cols):
    for k in ("gate8", "up8"):
        s[k] = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
        s[k + "_scale"] = torch.empty(rows, -(-cols // GROUP), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _scratch(s, nbytes):
    """The workspace that a program keeps from step to step."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_norms_fwd(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    L.liger_block_norm_fwd(s["z"], s["r"], s["h"], s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                           rstd_z=s["rstd_z"], rstd_h=s["rstd_h"], res_scale=c["res_scale"], block_scale=c["block_scale"],
                           eps=EPS)
    return {k: s[k] for k in ("h", "y", "rstd_z", "rstd_h")}


def _own_norms_bwd(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    if "ws" not in s:
        _scratch(s, L.liger_block_norm_bwd_workspace(c["rows"], c["cols"], c["gates"]))
    L.liger_block_norm_bwd(s["dh"], s["dy"], s["z"], s["h"], s["dr"], s["dz"], s["ws"], w_post=s["w_post"], gate=s["gate"],
                           w_pre=s["w_pre"], rstd_z=s["rstd_z"], rstd_h=s["rstd_h"], dw_post=s["dw_post"],
                           dgate=s["dgate"], dw_pre=s["dw_pre"], res_scale=c["res_scale"], block_scale=c["block_scale"])
    return {k: s[k] for k in ("dr", "dz", "dw_post", "dgate", "dw_pre")}


def _own_swiglu8(s):
    import transformer_rmsnorm_fwd_gb300 as L
    kept = (s["gate8"], s["gate8_scale"], s["up8"], s["up8_scale"])
    L.liger_swiglu_fwd_ckpt8(s["gate"], s["up"], s["y"], *kept)
    L.liger_swiglu_bwd_ckpt8(s["dy"], *kept, s["dgate"], s["dup"])
    return {k: s[k] for k in ("y", "dgate", "dup")}


def _own_linear_swiglu8(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    if "ws" not in s:
        _scratch(s, L.liger_fused_linear_swiglu_workspace(c["tokens"], c["inter"]))
    kept = (s["gate8"], s["gate8_scale"], s["up8"], s["up8_scale"])
    L.liger_fused_linear_swiglu_fwd_ckpt8(s["X"], s["Wg"], s["Wu"], s["out"], *kept)
    L.liger_fused_linear_swiglu_bwd_ckpt8(s["X"], s["Wg"], s["Wu"], s["dH"], *kept, s["dX"], s["dWg"], s["dWu"], s["ws"])
    return {k: s[k] for k in ("out", "dX", "dWg", "dWu")}


def _own_logp(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    if "ws" not in s:
        _scratch(s, L.liger_linear_logp_workspace(c["tokens"], c["hidden"], c["vocab"],
                                                  L.LIGER_BF16 if c["dtype"] == BF16 else L.LIGER_F32))
    L.liger_linear_logp_fwd(s["X"], s["W"], s["labels"], s["logp"], s["ws"], ignore_index=IGNORE)
    return {"logp": s["logp"]}


def _own_policy(s):
    import transformer_rmsnorm_fwd_gb300 as L
    c = s["case"]
    if "ws" not in s:
        _scratch(s, L.liger_linear_policy_workspace(c["tokens"], c["hidden"], c["vocab"], c["seqs"], 0,
                                                    L.LIGER_BF16 if c["dtype"] == BF16 else L.LIGER_F32))
    L.liger_linear_policy_fwd_bwd(s["X"], s["W"], s["labels"], s["old"], s["adv"], s["loss"], s["dX"], s["dW"], s["ws"],
                                  ref_logp=s["ref"], cu_seqlens=s["cu"], logp=s["logp"], stats=s["stats"],
                                  ignore_index=IGNORE, reduction=c["reduction"], eps_low=c["eps_low"],
                                  eps_high=c["eps_high"], beta=c["beta"])
    return {k: s[k] for k in ("loss", "dX", "dW", "logp", "stats")}


_OWN = {"norms_fwd": _own_norms_fwd, "norms_bwd": _own_norms_bwd, "swiglu8": _own_swiglu8,
        "linear_swiglu8": _own_linear_swiglu8, "logp": _own_logp, "policy": _own_policy}


# ------------------------------------------------------------------------------------------------ plain forms (32 bits)
def _gate_rows(gate, rows):
    """The gate of each row: gate row t // (rows / gates)."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0) if gate.shape[0] > 1 else gate.float()


def _plain_norms_fwd(s):
    c, dt = s["case"], s["z"].dtype
    z, r = s["z"].float(), s["r"].float()
    out = {"rstd_z": None, "rstd_h": None, "y": None}
    if c["post"]:
        out["rstd_z"] = torch.rsqrt(z.square().mean(1) + EPS)
        z = z * out["rstd_z"][:, None] * s["w_post"].float()
    if c["gates"]:
        z = z * _gate_rows(s["gate"], c["rows"])
    h = c["res_scale"] * r + c["block_scale"] * z
    out["h"] = h.to(dt)
    if c["pre"]:
        out["rstd_h"] = torch.rsqrt(h.square().mean(1) + EPS)
        out["y"] = (h * out["rstd_h"][:, None] * s["w_pre"].float()).to(dt)
    return out


def _plain_norms_bwd(s):
    c, dt = s["case"], s["z"].dtype
    z, h = s["z"].float(), s["h"].float()
    G, H = c["gates"], c["cols"]
    out = {"dw_post": None, "dgate": None, "dw_pre": None}
    D = s["dh"].float() if s["dh"] is not None else torch.zeros_like(h)
    if c["pre"]:
        dy, rh = s["dy"].float(), s["rstd_h"][:, None]
        hn = h * rh
        u = dy * s["w_pre"].float()
        out["dw_pre"] = (dy * hn).sum(0).to(dt)
        D = D + rh * (u - hn * (u * hn).mean(1, keepdim=True))
    out["dr"] = (c["res_scale"] * D).to(dt)
    D = D * c["block_scale"]
    rz = s["rstd_z"][:, None] if c["post"] else 1.0
    zn = z * rz
    if G:
        p = zn * s["w_post"].float() if c["post"] else zn
        out["dgate"] = (D * p).view(G, -1, H).sum(1).to(dt)
        D = D * _gate_rows(s["gate"], c["rows"])
    if c["post"]:
        out["dw_post"] = (D * zn).sum(0).to(dt)
        D = D * s["w_post"].float()
        D = rz * (D - zn * (D * zn).mean(1, keepdim=True))
    out["dz"] = D.to(dt)
    return out


def _plain_checkpoint(x):
    """What an 8-bit checkpoint gives back: multiples, up to 127, of a power of two for each GROUP columns of a row."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % GROUP)).view(rows, -1, GROUP)
    top = x.abs().amax(2, keepdim=True)
    _, e = torch.frexp(top)                               # top = m 2^e, 1/2 <= m < 1
    step = torch.ldexp(torch.ones_like(top), e - 7)
    back = (x / step).round().clamp(-127, 127) * step
    return torch.where(top > 0, back, 0.0).view(rows, -1)[:, :cols]


def _plain_swiglu_grads(g, u, dy):
    sig = 1.0 / (1.0 + torch.exp(-g))
    return dy * u * sig * (1.0 + g * (1.0 - sig)), dy * g * sig


def _plain_swiglu8(s):
    dt = s["gate"].dtype
    g, u = s["gate"].float(), s["up"].float()
    y = g / (1.0 + torch.exp(-g)) * u
    dg, du = _plain_swiglu_grads(_plain_checkpoint(g), _plain_checkpoint(u), s["dy"].float())
    return {"y": y.to(dt), "dgate": dg.to(dt), "dup": du.to(dt)}


def _plain_linear_swiglu8(s):
    dt = s["X"].dtype
    X, Wg, Wu = s["X"].float(), s["Wg"].float(), s["Wu"].float()
    g, u = X @ Wg.T, X @ Wu.T
    out = g / (1.0 + torch.exp(-g)) * u
    dg, du = _plain_swiglu_grads(_plain_checkpoint(g), _plain_checkpoint(u), s["dH"].float())
    return {"out": out.to(dt), "dX": (dg @ Wg + du @ Wu).to(dt), "dWg": (dg.T @ X).to(dt), "dWu": (du.T @ X).to(dt)}


def _plain_label_logp(z, labels):
    """Label log-probabilities (0 where masked) and softmax of logits."""
    e = z - z.amax(1, keepdim=True)
    y = labels.clamp(min=0)[:, None]
    zy = e.gather(1, y)[:, 0]
    e = e.exp_()
    total = e.sum(1)
    return torch.where(labels != IGNORE, zy - total.log(), 0.0), e, total


def _plain_logp(s):
    logp, _, _ = _plain_label_logp(s["X"].float() @ s["W"].float().T, s["labels"])
    return {"logp": logp}


def _plain_policy(s):
    c, dt, labels = s["case"], s["X"].dtype, s["labels"]
    T, B = c["tokens"], c["seqs"]
    X, W = s["X"].float(), s["W"].float()
    logp, e, total = _plain_label_logp(X @ W.T, labels)
    valid = labels != IGNORE
    seq = torch.searchsorted(s["cu"], torch.arange(T, dtype=torch.int32, device=X.device), right=True).sub(1).clamp(0, B - 1)
    n_seq = torch.zeros(B, device=X.device).index_add(0, seq, valid.float())
    n = valid.sum().clamp(min=1)
    if c["reduction"] == "token_mean":
        weight = valid / n
    elif c["reduction"] == "seq_mean":
        weight = valid / (B * n_seq.clamp(min=1))[seq]
    else:
        weight = valid.float()
    A = s["adv"][seq]
    ratio = torch.where(valid, torch.exp(logp - s["old"]), 1.0)
    held = ratio.clamp(1 - c["eps_low"], 1 + c["eps_high"])
    clipped = valid & (((A > 0) & (ratio > 1 + c["eps_high"])) | ((A < 0) & (ratio < 1 - c["eps_low"])))
    term = -torch.minimum(ratio * A, held * A)
    slope = -torch.where(clipped, 0.0, ratio * A)
    kl = torch.zeros_like(term)
    if c["beta"]:
        d = torch.where(valid, s["ref"] - logp, 0.0)
        kl = torch.exp(d) - d - 1.0
        term = term + c["beta"] * kl
        slope = slope + c["beta"] * (1.0 - torch.exp(d))
    loss = (weight.double() * term.double()).sum().float().view(1)
    stats = torch.stack([torch.where(valid, kl, 0.0).double().sum() / n, clipped.sum() / n.double()]).float()
    coef = weight * slope
    D = e.mul_((-coef / total)[:, None])
    D.scatter_add_(1, labels.clamp(min=0)[:, None], coef[:, None])
    return {"loss": loss, "dX": (D @ W).to(dt), "dW": (D.T @ X).to(dt), "logp": logp, "stats": stats}


_PLAIN = {"norms_fwd": _plain_norms_fwd, "norms_bwd": _plain_norms_bwd, "swiglu8": _plain_swiglu8,
          "linear_swiglu8": _plain_linear_swiglu8, "logp": _plain_logp, "policy": _plain_policy}


# ------------------------------------------------------------------------------------------------ least work
def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == BF16 else 4
    if op in ("norms_fwd", "norms_bwd"):
        n, H = case["rows"] * case["cols"], case["cols"]
        vectors = H * (case["post"] + case["pre"] + case["gates"])
        if op == "norms_fwd":
            return {"bytes": size * (n * (3 + case["pre"]) + vectors) + 4 * case["rows"] * (case["post"] + case["pre"]),
                    "flops": 10.0 * n}
        reads_z = case["post"] or case["gates"] > 0
        grads = case["pre"] + (case["grad_h"] or not case["pre"])
        return {"bytes": size * (n * (2 + grads + reads_z + case["pre"]) + 2 * vectors)
                + 4 * case["rows"] * (case["post"] + case["pre"]), "flops": 25.0 * n}
    if op == "swiglu8":
        n = case["rows"] * case["cols"]
        kept = 2 * (n + case["rows"] * -(-case["cols"] // GROUP))
        return {"bytes": 6 * size * n + 2 * kept, "flops": 30.0 * n}
    if op == "linear_swiglu8":
        T, H, I = case["tokens"], case["hidden"], case["inter"]
        kept = 2 * (T * I + T * -(-I // GROUP))
        return {"bytes": size * (2 * T * H + T * H + 2 * T * I + 6 * I * H) + 2 * kept, "flops": 12.0 * T * H * I}
    T, H, V = case["tokens"], case["hidden"], case["vocab"]
    n = sum(_layout(case)[1])
    if op == "logp":
        return {"bytes": size * (n * H + V * H) + 12 * T, "flops": 2.0 * n * H * V}
    return {"bytes": size * (n * H + T * H + 2 * V * H) + 20 * T, "flops": 6.0 * n * H * V}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return _EXACT[case["op"]](case, d)


def _each(case, gate):
    index = torch.arange(case["rows"], device="cuda") // (case["rows"] // case["gates"])
    return gate[index]


def _exact_norms_fwd(c, d):
    p = d["z"]
    rz = rh = y = None
    if c["post"]:
        rz = 1 / torch.sqrt((p * p).sum(1) / c["cols"] + EPS)
        p = torch.einsum("th,t,h->th", p, rz, d["w_post"])
    if c["gates"]:
        p = p * _each(c, d["gate"])
    h = d["r"] * c["res_scale"] + p * c["block_scale"]
    if c["pre"]:
        rh = 1 / torch.sqrt((h * h).sum(1) / c["cols"] + EPS)
        y = torch.einsum("th,t,h->th", h, rh, d["w_pre"])
    return {"h": h, "y": y, "rstd_z": rz, "rstd_h": rh}


def _exact_norms_bwd(c, d):
    T, H = c["rows"], c["cols"]
    z, h = d["z"], d["h"]
    D = d["dh"] if d["dh"] is not None else torch.zeros_like(h)
    dw_pre = dw_post = dgate = None
    if c["pre"]:
        rh = d["rstd_h"]
        u = d["dy"] * d["w_pre"]
        D = D + u * rh[:, None] - h * (rh ** 3 * (u * h).sum(1) / H)[:, None]
        dw_pre = torch.einsum("th,th,t->h", d["dy"], h, rh)
    q = torch.full((T, H), c["block_scale"], dtype=torch.float64, device=z.device)
    if c["gates"]:
        q = q * _each(c, d["gate"])
    rz = d["rstd_z"] if c["post"] else torch.ones(T, dtype=torch.float64, device=z.device)
    S = D * z * rz[:, None]
    if c["gates"]:
        per = torch.zeros(c["gates"], H, dtype=torch.float64, device=z.device)
        per.index_add_(0, torch.arange(T, device=z.device) // (T // c["gates"]), S)
        dgate = per * c["block_scale"] * (d["w_post"] if c["post"] else 1.0)
    if c["post"]:
        dw_post = (q * S).sum(0)
        q = q * d["w_post"]
        dz = q * D * rz[:, None] - z * (rz ** 3 * (q * D * z).sum(1) / H)[:, None]
    else:
        dz = q * D
    return {"dr": D * c["res_scale"], "dz": dz, "dw_post": dw_post, "dgate": dgate, "dw_pre": dw_pre}


def _exact_checkpoint(x):
    out = torch.empty_like(x)
    for a in range(0, x.shape[1], GROUP):
        part = x[:, a:a + GROUP]
        top = part.abs().max(1).values
        step = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 6)[:, None]
        out[:, a:a + GROUP] = torch.clamp(torch.round(part / step), -127, 127) * step
    return out


def _exact_activation(g, u, dy):
    sig = torch.sigmoid(g)
    gq, uq = _exact_checkpoint(g), _exact_checkpoint(u)
    sq = torch.sigmoid(gq)
    return g * sig * u, dy * uq * (sq + gq * sq * (1 - sq)), dy * gq * sq


def _exact_swiglu8(c, d):
    y, dg, du = _exact_activation(d["gate"], d["up"], d["dy"])
    return {"y": y, "dgate": dg, "dup": du}


def _exact_linear_swiglu8(c, d):
    if 12 * c["tokens"] * c["hidden"] * c["inter"] > 1.2e13:
        return None
    X, Wg, Wu = d["X"], d["Wg"], d["Wu"]
    out, dg, du = _exact_activation(X @ Wg.T, X @ Wu.T, d["dH"])
    return {"out": out, "dX": dg @ Wg + du @ Wu, "dWg": dg.T @ X, "dWu": du.T @ X}


def _exact_logp(c, d):
    labels, logp = d["labels"], torch.zeros(c["tokens"], dtype=torch.float64, device="cuda")
    for t in torch.nonzero(labels != IGNORE)[:, 0].split(1024):
        z = d["X"][t] @ d["W"].T
        logp[t] = z.gather(1, labels[t, None])[:, 0] - torch.logsumexp(z, 1)
    return {"logp": logp}


def _exact_policy(c, d):
    X, W, labels = d["X"], d["W"], d["labels"]
    starts, valid = _layout(c)
    n = max(1, sum(valid))
    dX, dW = torch.zeros_like(X), torch.zeros_like(W)
    logp = _exact_logp(c, d)["logp"]
    loss, kl_sum, clips = 0.0, 0.0, 0
    for b in range(c["seqs"]):
        t = torch.tensor([i for i in range(starts[b], starts[b + 1]) if valid[i]], dtype=torch.int64, device="cuda")
        if not len(t):
            continue
        weight = {"token_mean": 1.0 / n, "seq_mean": 1.0 / (c["seqs"] * len(t)), "sum": 1.0}[c["reduction"]]
        A, r = float(d["adv"][b]), torch.exp(logp[t] - d["old"][t])
        stop = (r > 1 + c["eps_high"]) if A > 0 else (r < 1 - c["eps_low"]) if A < 0 else torch.zeros_like(r, dtype=torch.bool)
        edge = 1 + c["eps_high"] if A > 0 else 1 - c["eps_low"]
        term = -torch.where(stop, edge, r) * A
        slope = torch.where(stop, 0.0, -r * A)
        clips += int(stop.sum())
        if c["beta"]:
            gap = d["ref"][t] - logp[t]
            kl = torch.expm1(gap) - gap
            kl_sum += float(kl.sum())
            term, slope = term + c["beta"] * kl, slope - c["beta"] * torch.expm1(gap)
        loss += weight * float(term.sum())
        for at, k in zip(t.split(1024), (weight * slope).split(1024)):
            D = -torch.softmax(X[at] @ W.T, 1) * k[:, None]
            D[torch.arange(len(at), device="cuda"), labels[at]] += k
            dX[at] = D @ W
            dW += D.T @ X[at]
    one = torch.tensor([loss], dtype=torch.float64, device="cuda")
    stats = torch.tensor([kl_sum / n, clips / n], dtype=torch.float64, device="cuda")
    return {"loss": one, "dX": dX, "dW": dW, "logp": logp, "stats": stats}


_EXACT = {"norms_fwd": _exact_norms_fwd, "norms_bwd": _exact_norms_bwd, "swiglu8": _exact_swiglu8,
          "linear_swiglu8": _exact_linear_swiglu8, "logp": _exact_logp, "policy": _exact_policy}
