"""liger_linear_logp_fwd and liger_linear_policy_fwd_bwd against the definition in 64 bits, whose gradients come from
automatic differentiation: both GEMM paths, chunks, both forms (with and without the host wait), packed sequences with masked,
empty and missing tokens, every reduction, bad labels and sequences, capture in a CUDA graph.

The bounds.  A logit's products are exact in fp32 and its sum of H terms is off by at most H 2^-23 of the terms' sizes
(tensor-core sums round toward zero); the sum of exponentials adds 2^-20 (the hardware's exp2 2^-22 and up to a few hundred
adds), the final subtraction 2^-22 of |z| and lse.  eps_lp below is that for each token.  A change of lp by eps changes the
ratio r A and the KL's exp(d) by that share.  On the bf16 path P and D are each rounded to bf16 once (2^-8 each of the
softmax part), then the GEMMs add in fp32."""
import math

import pytest
import torch

from train_util import U32, check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IGN = -100


@pytest.fixture(scope="module")
def L(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as lib
    return lib


def _code(L, dt):
    return L.LIGER_F32 if dt == "f32" else L.LIGER_BF16


def _inputs(T, H, V, dt, starts, seed=0, masked=0.3, lo=0.2, hi=0.2):
    """A packed batch: starts[b] .. starts[b + 1] is sequence b; NaN stands in every masked place."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, H, device="cuda", generator=g).to(DT[dt])
    W = (torch.randn(V, H, device="cuda", generator=g) * 1.3 * H ** -0.5).to(DT[dt])
    z = X.double() @ W.double().T
    labels = torch.randint(0, V, (T,), device="cuda", generator=g)
    labels[torch.rand(T, device="cuda", generator=g) < masked] = IGN
    valid = labels != IGN
    valid[:starts[0]] = False
    valid[starts[-1]:] = False
    lp = torch.log_softmax(z, 1).gather(1, labels.clamp(min=0)[:, None])[:, 0]
    d = 0.25 * torch.randn(T, device="cuda", generator=g, dtype=torch.float64)
    for e in (math.log(1 - lo) if lo < 1 else -50.0, math.log(1 + hi)):
        d = torch.where((d - e).abs() < 0.01, e + 0.02, d)      # not at the edge, where the gradient jumps
    nan = float("nan")
    old = torch.where(valid, lp - d, nan).float()
    ref = torch.where(valid, lp + 0.5 * torch.randn(T, device="cuda", generator=g, dtype=torch.float64), nan).float()
    adv = torch.randn(len(starts) - 1, device="cuda", generator=g)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    # where a token lies in no sequence its label may be anything in range: it is not read as one
    return dict(X=X, W=W, labels=labels, valid=valid, old=old, ref=ref, adv=adv, cu=cu, starts=starts)


def _ref(i, reduction, lo, hi, beta, gs, adv_per_token=False):
    X, W = i["X"].double().requires_grad_(), i["W"].double().requires_grad_()
    T, V = X.shape[0], W.shape[0]
    valid, B = i["valid"], len(i["starts"]) - 1
    at = torch.nonzero(valid)[:, 0]
    seq = torch.searchsorted(i["cu"].long(), at, right=True) - 1
    n_seq = torch.bincount(seq, minlength=B).double()
    w = {"token_mean": torch.full((len(at),), 1.0 / max(1, len(at))), "sum": torch.ones(len(at))}.get(reduction)
    w = (1.0 / (B * n_seq[seq])) if w is None else w.double().cuda()
    z = X[at] @ W.T
    lp = torch.log_softmax(z, 1).gather(1, i["labels"][at][:, None])[:, 0]
    A = (i["adv"][at] if adv_per_token else i["adv"][seq]).double()
    r = torch.exp(lp - i["old"][at].double())
    pol = -torch.minimum(r * A, r.clamp(1 - lo, 1 + hi) * A)
    d = i["ref"][at].double() - lp
    kl = torch.exp(d) - d - 1
    loss = (w * (pol + beta * kl)).sum()
    dX, dW = torch.autograd.grad(loss, (X, W))
    with torch.no_grad():
        clip = ((A > 0) & (r > 1 + hi)) | ((A < 0) & (r < 1 - lo))
        logp = torch.zeros(T, dtype=torch.float64, device="cuda")
        logp[at] = lp
        xw = (X[at].abs() @ W.abs().T).amax(1) if len(at) else torch.zeros(0, device="cuda")
        eps = X.shape[1] * 2.0 ** -23 * xw + 2.0 ** -20 + 2.0 ** -22 * (z.gather(1, i["labels"][at][:, None])[:, 0].abs() * 2 + lp.abs())
        eps_all = torch.zeros(T, dtype=torch.float64, device="cuda")
        eps_all[at] = eps
        # sizes: |dl/dlp| and its change with lp are within w (|r A| + beta (1 + e^d))
        size = w * ((r * A).abs() * ~clip + abs(beta) * (1 + torch.exp(d)))
        p = torch.softmax(z, 1)
        soft = abs(gs) * size[:, None] * p
        hot = abs(gs) * size
        y = i["labels"][at]
        mX = torch.zeros_like(X)
        mX[at] = soft @ W.abs() + hot[:, None] * W[y].abs()
        mW = soft.T @ X[at].abs()
        mW.index_add_(0, y, hot[:, None] * X[at].abs())
        e = float(eps.max()) if len(at) else 0.0
        loss_off = float((size * eps).sum()) + 8 * U32 * float((w * (pol.abs() + abs(beta) * (kl + 1e-3))).sum())
        n = max(1, len(at))
        stats = (float(kl.sum()) / n, float(clip.sum()) / n)
        kl_off = float(((1 + torch.exp(d)) * eps).sum()) / n + 8 * U32 * stats[0]
    return dict(loss=float(loss.detach()), dX=gs * dX, dW=gs * dW, logp=logp, eps=eps_all, mX=mX, mW=mW, e=e, loss_off=loss_off,
                stats=stats, kl_off=kl_off)


def _call(L, i, dt, reduction, lo, hi, beta, gs, wait=True, chunk=0, adv_per_token=False, ref=True, want=(True, True),
          cu=True, ws=None):
    T, H = i["X"].shape
    V, B = i["W"].shape[0], len(i["starts"]) - 1 if cu else 1
    if ws is None:
        ws = torch.full((L.liger_linear_policy_workspace(T, H, V, B, chunk, _code(L, dt)),), 255, dtype=torch.uint8, device="cuda")
    o = dict(loss=torch.full((1,), 7.0, device="cuda"), stats=torch.full((2,), 7.0, device="cuda"),
             logp=torch.full((T,), 7.0, device="cuda"), dX=torch.full_like(i["X"], 7.0) if want[0] else None,
             dW=torch.full_like(i["W"], 7.0) if want[1] else None)
    L.liger_linear_policy_fwd_bwd(i["X"], i["W"], i["labels"], i["old"], i["adv"], o["loss"], o["dX"], o["dW"], ws,
                                  ref_logp=i["ref"] if ref else None, cu_seqlens=i["cu"] if cu else None, logp=o["logp"],
                                  stats=o["stats"], reduction=reduction, eps_low=lo, eps_high=hi, beta=beta, grad_scale=gs,
                                  adv_per_token=adv_per_token, chunk=chunk, wait=wait)
    return o


def _compare(o, r, i, dt, tc):
    T, H = i["X"].shape
    V = i["W"].shape[0]
    assert bool(((o["logp"].double() - r["logp"]).abs() <= r["eps"])[i["valid"]].all())
    assert bool((o["logp"][~i["valid"]] == 0).all())
    assert abs(float(o["loss"]) - r["loss"]) <= r["loss_off"] + 2 * U32 * abs(r["loss"]) + 1e-30
    assert abs(float(o["stats"][0]) - r["stats"][0]) <= r["kl_off"] + 1e-12
    assert abs(float(o["stats"][1]) - r["stats"][1]) <= 2 * U32
    low = 2 * 2.0 ** 16 * 1.01 if tc else 0        # P and D rounded to bf16
    # exp(z - lse): |z - lse| 2^-23 of argument rounding, the lp error in z and lse, in c once more
    common = low + 3 * r["e"] * 2 ** 24 + 200
    if o["dX"] is not None:
        check(o["dX"], r["dX"], r["mX"], common + 2 * V ** 0.5 + 2 * 256, "dX") if tc else check(o["dX"], r["dX"], r["mX"], common + V, "dX")
        assert bool((o["dX"][~i["valid"]].view(torch.int16 if dt == "bf16" else torch.int32) == 0).all())
    if o["dW"] is not None:
        check(o["dW"], r["dW"], r["mW"], common + 2 * T, "dW")


CASES = [   # T, H, V, dtype, sequence starts, chunk
    (1, 64, 256, "bf16", [0, 1], 0), (1, 8, 5, "f32", [0, 1], 0), (37, 64, 300, "bf16", [0, 10, 10, 36], 0),
    (300, 320, 2037, "bf16", [0, 1, 150, 151, 290], 0), (300, 320, 2037, "bf16", [0, 300], 128),
    (257, 136, 777, "bf16", [3, 80, 200, 257], 0), (130, 50, 300, "bf16", [0, 60, 130], 0),     # H not a multiple of 8: fp32 path
    (129, 72, 515, "f32", [0, 60, 60, 129], 0), (200, 33, 100, "f32", [0, 100, 190], 64),
    (600, 64, 66536, "bf16", [0, 300, 600], 0),         # dX over two slabs of the vocabulary
    (9000, 64, 300, "bf16", [0, 4000, 9000], 16384),    # several label-sort segments in one chunk
]


@pytest.mark.parametrize("T,H,V,dt,starts,chunk", CASES)
@pytest.mark.parametrize("wait", [True, False])
def test_policy(L, T, H, V, dt, starts, chunk, wait):
    tc = dt == "bf16" and H % 8 == 0
    for n, (reduction, lo, hi, beta, gs, masked) in enumerate([
            ("seq_mean", 0.2, 0.28, 0.05, 1.0, 0.3), ("token_mean", 0.2, 0.2, 0.0, 0.5, 0.0), ("sum", 1.0, 0.0, 0.3, -2.0, 0.6)]):
        i = _inputs(T, H, V, dt, starts, seed=n + T, masked=masked if T > 1 else 0.0, lo=lo, hi=hi)
        r = _ref(i, reduction, lo, hi, beta, gs)
        o = _call(L, i, dt, reduction, lo, hi, beta, gs, wait, chunk)
        _compare(o, r, i, dt, tc)


@pytest.mark.parametrize("T,H,V", [
    (2600, 2048, 66536),    # 88 dX tiles: a full round and 12 split tiles, over two slabs of the vocabulary
    (2600, 2048, 3000),     # the same in one launch
    (20, 4096, 70000),      # 16 tiles split over all pairs
    (130, 520, 2100),       # 3 tiles; k ranges that do not divide the k-blocks
])
def test_policy_split_dx(L, T, H, V):
    i = _inputs(T, H, V, "bf16", [0, T // 2, T], seed=T, masked=0.0)
    r = _ref(i, "seq_mean", 0.2, 0.2, 0.05, 1.0)
    o = _call(L, i, "bf16", "seq_mean", 0.2, 0.2, 0.05, 1.0)
    _compare(o, r, i, "bf16", True)
    again = _call(L, i, "bf16", "seq_mean", 0.2, 0.2, 0.05, 1.0, wait=False)
    for k in o:
        assert torch.equal(o[k], again[k]), k


def test_forms_agree_and_repeat(L):
    """No masked token: both forms are the same bits; a second run is the same bits; one output alone equals both."""
    i = _inputs(500, 128, 1000, "bf16", [0, 200, 500], masked=0.0)
    a = _call(L, i, "bf16", "seq_mean", 0.2, 0.2, 0.1, 1.0)
    for kw in (dict(wait=False), dict(), dict(want=(True, False)), dict(want=(False, True)), dict(want=(False, False))):
        b = _call(L, i, "bf16", "seq_mean", 0.2, 0.2, 0.1, 1.0, **kw)
        for k in a:
            assert b[k] is None or torch.equal(a[k], b[k]), (kw, k)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_sequence_and_token_advantages(L, dt):
    T, H, V = 140, 64, 400
    i = _inputs(T, H, V, dt, [0, T], seed=4)
    i["adv"] = torch.where(i["valid"], torch.randn(T, device="cuda"), float("nan"))
    i["adv"][3] = 0.0
    r = _ref(i, "token_mean", 0.2, 0.2, 0.02, 1.0, adv_per_token=True)
    _compare(_call(L, i, dt, "token_mean", 0.2, 0.2, 0.02, 1.0, adv_per_token=True, cu=False), r, i, dt, dt == "bf16")


def test_without_reference_policy(L):
    i = _inputs(100, 64, 300, "bf16", [0, 40, 100], seed=8)
    r = _ref(i, "token_mean", 0.2, 0.2, 0.0, 1.0)
    o = _call(L, i, "bf16", "token_mean", 0.2, 0.2, 0.0, 1.0, ref=False)
    assert float(o["stats"][0]) == 0.0
    r["stats"], r["kl_off"] = (0.0, r["stats"][1]), 0.0
    _compare(o, r, i, "bf16", True)


def test_kl_of_close_policies(L):
    """kl of d near 0 keeps its relative precision (d^2 / 2): the reference equals the policy but for 1e-3."""
    i = _inputs(64, 64, 300, "f32", [0, 64], masked=0.0, seed=2)
    z = i["X"].double() @ i["W"].double().T
    lp = torch.log_softmax(z, 1).gather(1, i["labels"][:, None])[:, 0]
    i["ref"] = (lp + 1e-3).float()
    o = _call(L, i, "f32", "token_mean", 0.2, 0.2, 1.0, 1.0)
    d = i["ref"].double() - o["logp"].double()      # as the kernel sees it
    assert abs(float(o["stats"][0]) / float((torch.expm1(d) - d).mean()) - 1) < 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("wait", [True, False])
def test_nothing_valid(L, dt, wait):
    i = _inputs(70, 64, 300, dt, [0, 30, 70], masked=2.0)
    o = _call(L, i, dt, "seq_mean", 0.2, 0.2, 0.1, 1.0, wait)
    assert float(o["loss"]) == 0.0 and bool((o["stats"] == 0).all()) and bool((o["logp"] == 0).all())
    assert bool((o["dX"] == 0).all()) and bool((o["dW"] == 0).all())


def test_no_tokens(L):
    X, W = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.randn(300, 64, device="cuda").to(torch.bfloat16)
    e = torch.empty(0, device="cuda")
    lab = torch.empty(0, dtype=torch.int64, device="cuda")
    for wait in (True, False):
        loss, dW = torch.full((1,), 7.0, device="cuda"), torch.full_like(W, 7.0)
        ws = torch.empty(L.liger_linear_policy_workspace(0, 64, 300, 1), dtype=torch.uint8, device="cuda")
        L.liger_linear_policy_fwd_bwd(X, W, lab, e, torch.zeros(1, device="cuda"), loss, torch.empty_like(X), dW, ws, wait=wait)
        assert float(loss) == 0.0 and bool((dW == 0).all())
        L.liger_linear_logp_fwd(X, W, lab, e, ws, wait=wait)


def test_bad_labels_and_sequences(L):
    i = _inputs(200, 64, 300, "bf16", [0, 80, 200], masked=0.2)
    args = ("bf16", "token_mean", 0.2, 0.2, 0.1, 1.0)
    bad = dict(i, labels=i["labels"].clone())
    bad["labels"][5] = 300
    fixed = dict(i, labels=i["labels"].clone())
    fixed["labels"][5] = IGN
    with pytest.raises(L.LigerError) as e:
        _call(L, bad, *args)
    assert e.value.status == -5
    o, f = _call(L, bad, *args, wait=False), _call(L, fixed, *args, wait=False)
    assert math.isnan(float(o["loss"])) and bool(torch.isnan(o["stats"]).all())
    assert torch.equal(o["dX"], f["dX"]) and torch.equal(o["dW"], f["dW"]) and not math.isnan(float(f["loss"]))
    for cu in ([0, 120, 100, 200][1:], [-1, 80, 200], [0, 80, 201], [0, 2 ** 31 - 1, 200]):
        odd = dict(i, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        with pytest.raises(L.LigerError) as e:
            _call(L, odd, *args)
        assert e.value.status == -2
        o = _call(L, odd, *args, wait=False)
        assert math.isnan(float(o["loss"])) and bool((o["dX"] == 0).all()) and bool((o["dW"] == 0).all())


@pytest.mark.parametrize("T,H,V,dt,chunk", [(50, 64, 300, "bf16", 0), (50, 64, 300, "bf16", 16), (600, 64, 300, "bf16", 0),
                                            (50, 33, 100, "f32", 0), (600, 33, 100, "f32", 128)])
def test_a_bad_label_leaves_the_outputs(L, T, H, V, dt, chunk):
    """The waiting forms write no output when the scan finds a bad label, and the next call on the workspace is not disturbed."""
    i = _inputs(T, H, V, dt, [0, T], seed=T, masked=0.2)
    ws = torch.empty(L.liger_linear_policy_workspace(T, H, V, 1, chunk, _code(L, dt)), dtype=torch.uint8, device="cuda")
    good = _call(L, i, dt, "sum", 0.2, 0.2, 0.1, 1.0, chunk=chunk, ws=ws)
    lab = i["labels"].clone()
    lab[T - 1] = V
    out = dict(loss=torch.full((1,), 7.0, device="cuda"), stats=torch.full((2,), 7.0, device="cuda"),
               logp=torch.full((T,), 7.0, device="cuda"), dX=torch.full_like(i["X"], 7.0), dW=torch.full_like(i["W"], 7.0))
    for _ in range(3):
        with pytest.raises(L.LigerError) as e:
            L.liger_linear_policy_fwd_bwd(i["X"], i["W"], lab, i["old"], i["adv"], out["loss"], out["dX"], out["dW"], ws,
                                          ref_logp=i["ref"], cu_seqlens=i["cu"], logp=out["logp"], stats=out["stats"],
                                          reduction="sum", beta=0.1, chunk=chunk)
        assert e.value.status == -5
        assert all(bool((v == 7).all()) for v in out.values())
    again = _call(L, i, dt, "sum", 0.2, 0.2, 0.1, 1.0, chunk=chunk, ws=ws)
    assert all(torch.equal(again[k], good[k]) for k in good)


def test_non_finite_inputs_reach_the_loss(L):
    """NaN at a valid token is not hidden; a ratio of infinity is held by the clip when A > 0."""
    i = _inputs(60, 64, 300, "f32", [0, 60], masked=0.0)
    i["adv"][0] = 1.0
    i["old"][7] = float("-inf")
    r = _call(L, i, "f32", "token_mean", 0.2, 0.2, 0.0, 1.0, ref=False)
    assert math.isfinite(float(r["loss"])) and bool((r["dX"][7] == 0).all())
    i["old"][9] = float("nan")
    r = _call(L, i, "f32", "token_mean", 0.2, 0.2, 0.0, 1.0, ref=False)
    assert math.isnan(float(r["loss"])) and bool(torch.isnan(r["dX"][9]).any()) and bool(torch.isfinite(r["dX"][8]).all())


@pytest.mark.parametrize("wait", [True, False])
@pytest.mark.parametrize("T,H,V,dt,masked,chunk", [(200, 64, 300, "bf16", 0.3, 0), (900, 128, 600, "bf16", 0.7, 0),
                                                   (900, 128, 600, "bf16", 0.05, 256), (9, 72, 1003, "bf16", 0.5, 0),
                                                   (8300, 64, 300, "bf16", 0.01, 8300), (77, 40, 300, "bf16", 0.4, 32),
                                                   (120, 33, 100, "f32", 0.4, 0), (120, 33, 100, "f32", 0.4, 50)])
def test_hidden_states_of_tokens_that_are_not_valid(L, T, H, V, dt, masked, chunk, wait):
    """Padding may hold anything: NaN and infinities in X at masked tokens and outside the sequences reach no output."""
    i = _inputs(T, H, V, dt, [2, T // 2, T - 3], seed=T, masked=masked)
    args = (dt, "seq_mean", 0.2, 0.2, 0.05, 1.0)
    clean = _call(L, i, *args, wait=wait, chunk=chunk)
    junk = i["X"].clone()
    junk[~i["valid"]] = float("nan")
    junk[0] = float("inf")
    got = _call(L, dict(i, X=junk), *args, wait=wait, chunk=chunk)
    for k, v in clean.items():
        assert torch.equal(got[k], v) and bool(torch.isfinite(v).all()), k
    out, ws = [], torch.empty(L.liger_linear_logp_workspace(T, H, V, _code(L, dt)), dtype=torch.uint8, device="cuda")
    for X in (i["X"], junk):
        logp = torch.full((T,), 7.0, device="cuda")
        lab = torch.where(i["valid"], i["labels"], IGN)
        L.liger_linear_logp_fwd(X, i["W"], lab, logp, ws, wait=wait)
        out.append(logp)
    assert torch.equal(*out) and bool(torch.isfinite(out[0]).all())


@pytest.mark.parametrize("wait", [True, False])
@pytest.mark.parametrize("T,H,V,dt", [(1, 64, 256, "bf16"), (1, 512, 5000, "bf16"), (300, 320, 2037, "bf16"), (77, 40, 300, "bf16"),
                                      (65, 33, 100, "f32"), (1, 3, 2, "f32"), (9000, 64, 300, "bf16"),
                                      (2, 128, 300, "bf16"), (3, 72, 1003, "bf16"), (4, 4096, 5001, "bf16"), (5, 256, 257, "bf16"),
                                      (8, 520, 70001, "bf16"), (9, 520, 2000, "bf16"), (6, 16384, 300, "bf16")])
def test_logp(L, T, H, V, dt, wait):
    for masked in (0.0, 0.4, 2.0):
        i = _inputs(T, H, V, dt, [0, T], seed=T, masked=masked)
        r = _ref(i, "sum", 0.2, 0.2, 0.0, 1.0)
        ws = torch.full((L.liger_linear_logp_workspace(T, H, V, _code(L, dt)),), 255, dtype=torch.uint8, device="cuda")
        logp = torch.full((T,), 7.0, device="cuda")
        L.liger_linear_logp_fwd(i["X"], i["W"], i["labels"], logp, ws, wait=wait)
        assert bool(((logp.double() - r["logp"]).abs() <= r["eps"])[i["valid"]].all())
        assert bool((logp[~i["valid"]] == 0).all())


@pytest.mark.parametrize("T,V", [(1, 300), (2, 5000), (3, 70001), (4, 300), (5, 300), (40, 5000)])
def test_logp_of_non_finite_rows_of_the_head(L, T, V):
    """A row of W whose logit is -inf has probability 0, wherever it stands; a NaN row makes every logp NaN."""
    i = _inputs(T, 64, V, "bf16", [0, T], seed=V, masked=0.0)
    i["X"][:, 5] = 1.0
    i["labels"].fill_(V // 2)
    ws = torch.empty(L.liger_linear_logp_workspace(T, 64, V), dtype=torch.uint8, device="cuda")
    for row in (0, 1, 2, 17, V - 1):
        W = i["W"].clone()
        W[row, 5] = float("-inf")
        keep = torch.arange(V, device="cuda") != row
        i2 = dict(i, W=W[keep], labels=i["labels"] - int(row < V // 2))
        i2["old"] = i2["ref"] = torch.zeros(T, device="cuda")
        r = _ref(i2, "sum", 0.2, 0.2, 0.0, 1.0)
        for value, wait in ((float("-inf"), True), (float("-inf"), False), (float("nan"), False)):
            W[row, 5] = value
            logp = torch.full((T,), 7.0, device="cuda")
            L.liger_linear_logp_fwd(i["X"], W, i["labels"], logp, ws, wait=wait)
            if value == value:
                assert bool(((logp.double() - r["logp"]).abs() <= r["eps"]).all()), row
            else:
                assert bool(torch.isnan(logp).all()), row


def test_logp_bad_label(L):
    i = _inputs(50, 64, 300, "bf16", [0, 50], masked=0.2)
    ws = torch.empty(L.liger_linear_logp_workspace(50, 64, 300), dtype=torch.uint8, device="cuda")
    good, logp = torch.empty(50, device="cuda"), torch.full((50,), 7.0, device="cuda")
    L.liger_linear_logp_fwd(i["X"], i["W"], i["labels"], good, ws, wait=False)
    lab = i["labels"].clone()
    lab[11] = -1
    with pytest.raises(L.LigerError) as e:
        L.liger_linear_logp_fwd(i["X"], i["W"], lab, logp, ws)
    assert e.value.status == -5 and bool((logp == 7).all())
    L.liger_linear_logp_fwd(i["X"], i["W"], lab, logp, ws, wait=False)
    rest = torch.arange(50, device="cuda") != 11
    assert math.isnan(float(logp[11])) and torch.equal(logp[rest], good[rest])


def test_policy_logp_is_logp(L):
    i = _inputs(400, 128, 3000, "bf16", [0, 100, 400], masked=0.3)
    o = _call(L, i, "bf16", "token_mean", 0.2, 0.2, 0.1, 1.0)
    ws = torch.empty(L.liger_linear_logp_workspace(400, 128, 3000), dtype=torch.uint8, device="cuda")
    logp = torch.empty(400, device="cuda")
    L.liger_linear_logp_fwd(i["X"], i["W"], i["labels"], logp, ws)
    assert torch.equal(logp, o["logp"])


def test_gradient_against_differences(L):
    """Slopes of the 64-bit loss along random directions."""
    i = _inputs(60, 24, 50, "f32", [0, 25, 60], masked=0.2, seed=5)
    o = _call(L, i, "f32", "seq_mean", 0.2, 0.2, 0.2, 1.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    for name, grad in (("X", "dX"), ("W", "dW")):
        v = torch.randn(i[name].shape, device="cuda", generator=g, dtype=torch.float64)
        one = [_ref(dict(i, **{name: i[name].double() + s * 1e-6 * v}), "seq_mean", 0.2, 0.2, 0.2, 1.0)["loss"] for s in (1, -1)]
        got = float((o[grad].double() * v).sum())
        size = float((o[grad].double().abs() * v.abs()).sum())
        assert abs(got - (one[0] - one[1]) / 2e-6) <= 1e-5 * size + 1e-8


def test_capture(L):
    """The forms without the host wait, captured and replayed on new inputs in the same buffers."""
    i, j = (_inputs(300, 128, 1000, "bf16", [0, 120, 290], seed=s) for s in (1, 2))
    ws = torch.empty(L.liger_linear_policy_workspace(300, 128, 1000, 2), dtype=torch.uint8, device="cuda")
    lws = torch.empty(L.liger_linear_logp_workspace(300, 128, 1000), dtype=torch.uint8, device="cuda")
    want = _call(L, j, "bf16", "seq_mean", 0.2, 0.2, 0.1, 1.0, wait=False)
    out = dict(loss=torch.zeros(1, device="cuda"), dX=torch.zeros_like(i["X"]), dW=torch.zeros_like(i["W"]),
               logp=torch.zeros(300, device="cuda"), stats=torch.zeros(2, device="cuda"))
    alone = torch.zeros(300, device="cuda")

    def step():
        L.liger_linear_policy_fwd_bwd(i["X"], i["W"], i["labels"], i["old"], i["adv"], out["loss"], out["dX"], out["dW"], ws,
                                      ref_logp=i["ref"], cu_seqlens=i["cu"], logp=out["logp"], stats=out["stats"],
                                      reduction="seq_mean", beta=0.1, wait=False)
        L.liger_linear_logp_fwd(i["X"], i["W"], i["labels"], alone, lws, wait=False)
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step()
    for k in ("X", "W", "labels", "old", "ref", "adv"):
        i[k].copy_(j[k])
    graph.replay()
    torch.cuda.synchronize()
    for k in out:
        assert torch.equal(out[k], want[k]), k
    # tokens behind the last sequence have a log-probability of their own, but no place in the loss
    inside = j["valid"]
    assert torch.equal(alone[inside], out["logp"][inside])


def test_refusals(L):
    i = _inputs(20, 64, 300, "bf16", [0, 20])
    ws = torch.empty(L.liger_linear_policy_workspace(20, 64, 300, 1), dtype=torch.uint8, device="cuda")
    loss, dX, dW = torch.empty(1, device="cuda"), torch.empty_like(i["X"]), torch.empty_like(i["W"])
    args = (i["X"], i["W"], i["labels"], i["old"], i["adv"], loss, dX, dW, ws)
    with pytest.raises(L.LigerError) as e:      # beta without ref_logp
        L.liger_linear_policy_fwd_bwd(*args, beta=0.1)
    assert e.value.status == -1
    with pytest.raises(L.LigerError) as e:
        L.liger_linear_policy_fwd_bwd(*args, eps_low=1.5)
    assert e.value.status == -2
    with pytest.raises(L.LigerError) as e:
        L.liger_linear_policy_fwd_bwd(*args[:-1], ws[:-256])
    assert e.value.status == -6
    with pytest.raises(KeyError):
        L.liger_linear_policy_fwd_bwd(*args, reduction="mean")
    with pytest.raises(ValueError):             # one advantage for 20 tokens
        L.liger_linear_policy_fwd_bwd(*args, adv_per_token=True)
    with pytest.raises(TypeError):
        L.liger_linear_policy_fwd_bwd(*args, cu_seqlens=i["cu"].long())
    with pytest.raises(TypeError):
        L.liger_linear_logp_fwd(i["X"], i["W"].float(), i["labels"], i["old"], ws)
    with pytest.raises(TypeError):
        L.liger_linear_logp_fwd(i["X"], i["W"], i["labels"].int(), i["old"], ws)
