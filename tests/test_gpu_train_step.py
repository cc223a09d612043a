"""The post-training operators as one policy step of a small decoder: block norms around an MLP with 8-bit checkpoints, the
policy loss on the head; gradients of every weight against 64-bit automatic differentiation; the step on another stream,
captured in CUDA graphs (two at once), from several threads; tensors past 2^31 elements; refusals about devices."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-6
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as lib
    return lib


class Step:
    """One layer's tail and the head: r, z -> norms -> MLP -> norms -> policy loss, and back."""

    def __init__(self, L, T=384, H=256, I=544, V=1000, seed=0, beta=0.05):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s, std=1.0, mean=0.0):
            return (torch.randn(*s, device="cuda", generator=g) * std + mean).to(BF)
        self.L, self.dims, self.beta = L, (T, H, I, V), beta
        self.starts = [0, T // 3, T // 3, T - 7]
        p = self.p = {"z0": rnd(T, H), "r0": rnd(T, H)}
        for k in ("a", "b"):
            p["post_" + k], p["pre_" + k], p["gate_" + k] = (rnd(H, std=0.1, mean=1.0) for _ in range(3))
        p["Wg"], p["Wu"] = rnd(I, H, std=H ** -0.5), rnd(I, H, std=H ** -0.5)
        p["Wd"], p["W"] = rnd(H, I, std=I ** -0.5), rnd(V, H, std=1.3 * H ** -0.5)
        lab = torch.randint(0, V, (T,), device="cuda", generator=g)
        lab[torch.rand(T, device="cuda", generator=g) < 0.25] = -100
        self.labels = lab
        self.cu = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.adv = torch.randn(3, device="cuda", generator=g)
        # old and reference log-probabilities near the model's, away from the clip's edges (a bf16 step
        # of the hidden states moves a ratio by a few per cent, so "near" is ratios of 1 within 5 %, or 2)
        lp = self.reference(grad=False)
        far = torch.rand(T, device="cuda", generator=g) < 0.3
        d = torch.where(far, 0.7, 0.02 * torch.randn(T, device="cuda", generator=g)).double()
        self.old, self.ref = (lp - d).float(), (lp + 0.2).float()
        b = self.b = {}
        for k, s in (("h1", (T, H)), ("y1", (T, H)), ("m", (T, I)), ("h2", (T, H)), ("y2", (T, H)), ("dy2", (T, H)),
                     ("dh1", (T, H)), ("dz1", (T, H)), ("dy1", (T, H)), ("dz0", (T, H)), ("dr0", (T, H))):
            b[k] = torch.empty(s, device="cuda", dtype=BF)
        for k in p:
            if k not in ("z0", "r0"):
                b["d" + k] = torch.empty_like(p[k])
        for k in ("rz1", "rh1", "rz2", "rh2"):
            b[k] = torch.empty(T, device="cuda")
        b["kept"] = (*L.liger_ckpt8_empty(T, I), *L.liger_ckpt8_empty(T, I))
        b["loss"] = torch.empty(1, device="cuda")

        def ws(n):
            return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        b["ws_n"], b["ws_m"] = ws(L.liger_block_norm_bwd_workspace(T, H, 1)), ws(L.liger_fused_linear_swiglu_workspace(T, I))
        b["ws_p"] = ws(L.liger_linear_policy_workspace(T, H, V, 3))

    def run(self, wait=False):
        L, p, b = self.L, self.p, self.b
        L.liger_block_norm_fwd(p["z0"], p["r0"], b["h1"], b["y1"], p["post_a"], p["gate_a"], p["pre_a"], b["rz1"], b["rh1"],
                               eps=EPS)
        L.liger_fused_linear_swiglu_fwd_ckpt8(b["y1"], p["Wg"], p["Wu"], b["m"], *b["kept"])
        b["z1"] = b["m"] @ p["Wd"].T
        L.liger_block_norm_fwd(b["z1"], b["h1"], b["h2"], b["y2"], p["post_b"], p["gate_b"], p["pre_b"], b["rz2"], b["rh2"],
                               res_scale=0.9, block_scale=0.7, eps=EPS)
        L.liger_linear_policy_fwd_bwd(b["y2"], p["W"], self.labels, self.old, self.adv, b["loss"], b["dy2"], b["dW"],
                                      b["ws_p"], ref_logp=self.ref, cu_seqlens=self.cu, reduction="seq_mean",
                                      beta=self.beta, wait=wait)
        L.liger_block_norm_bwd(None, b["dy2"], b["z1"], b["h2"], b["dh1"], b["dz1"], b["ws_n"], p["post_b"], p["gate_b"],
                               p["pre_b"], b["rz2"], b["rh2"], b["dpost_b"], b["dgate_b"], b["dpre_b"], 0.9, 0.7)
        torch.matmul(b["dz1"].T, b["m"], out=b["dWd"])
        b["dm"] = b["dz1"] @ p["Wd"]
        L.liger_fused_linear_swiglu_bwd_ckpt8(b["y1"], p["Wg"], p["Wu"], b["dm"], *b["kept"], b["dy1"], b["dWg"], b["dWu"],
                                              b["ws_m"])
        L.liger_block_norm_bwd(b["dh1"], b["dy1"], p["z0"], b["h1"], b["dr0"], b["dz0"], b["ws_n"], p["post_a"], p["gate_a"],
                               p["pre_a"], b["rz1"], b["rh1"], b["dpost_a"], b["dgate_a"], b["dpre_a"])

    def grads(self):
        return {k: self.b["d" + k] for k in self.p}

    def reference(self, grad=True):
        """The loss's gradients in 64 bits, the MLP's backward from g and u as the 8-bit format gives them back."""
        p = {k: v.double().requires_grad_(grad) for k, v in self.p.items()}
        T = self.dims[0]

        def norms(z, r, k, a, b):
            q = z * (z.square().mean(1, keepdim=True) + EPS).rsqrt() * p["post_" + k] * p["gate_" + k]
            h = a * r + b * q
            return h, h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * p["pre_" + k]
        h1, y1 = norms(p["z0"], p["r0"], "a", 1.0, 1.0)
        m = _Act.apply(y1 @ p["Wg"].T, y1 @ p["Wu"].T)
        _, y2 = norms(m @ p["Wd"].T, h1, "b", 0.9, 0.7)
        lp_all = torch.log_softmax(y2 @ p["W"].T, 1).gather(1, self.labels.clamp(min=0)[:, None])[:, 0]
        if not grad:
            return lp_all
        loss = 0.0
        for s in range(3):
            t = torch.arange(self.starts[s], self.starts[s + 1], device="cuda")
            t = t[self.labels[t] != -100]
            if not len(t):
                continue
            lp, A = lp_all[t], self.adv[s].double()
            r = torch.exp(lp - self.old[t].double())
            d = self.ref[t].double() - lp
            loss = loss + (-torch.minimum(r * A, r.clamp(0.8, 1.2) * A) + self.beta * (torch.exp(d) - d - 1)).sum() / (3 * len(t))
        return dict(zip(p, torch.autograd.grad(loss, list(p.values())))), float(loss.detach())


class _Act(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, u):
        def back(x):
            v = torch.nn.functional.pad(x, (0, -x.shape[1] % 32)).view(x.shape[0], -1, 32)
            step = torch.exp2(torch.floor(torch.log2(v.abs().amax(2, keepdim=True))) - 6)
            return ((v / step).round().clamp(-127, 127) * step).reshape(x.shape[0], -1)[:, :x.shape[1]]
        ctx.save_for_backward(back(g), back(u))
        return g * torch.sigmoid(g) * u

    @staticmethod
    def backward(ctx, d):
        g, u = ctx.saved_tensors
        s = torch.sigmoid(g)
        return d * u * s * (1 + g * (1 - s)), d * g * s


def test_gradients_of_a_step(L):
    """Up to 13 tensors between the inputs and a gradient are rounded to bf16 (h, y, m, z, h, y forward; dy, dz, dh, dm,
    dG and dU, dy, dz backward), each 2^-8 of its values at most, and a softmax weight, a ratio and a normalised row pass a
    relative error on with a factor near 1: 13 2^-8 of a gradient's norm."""
    st = Step(L)
    for wait in (True, False):
        st.run(wait)
        want, loss = st.reference()
        for k, g in st.grads().items():
            rel = float((g.double() - want[k]).norm() / want[k].norm())
            assert rel <= 13 * 2.0 ** -8, (k, rel)
        assert abs(float(st.b["loss"]) - loss) <= 13 * 2.0 ** -8 * max(abs(loss), float(st.adv.abs().mean()))


def _snapshot(st):
    return {k: v.clone() for k, v in {**st.grads(), "loss": st.b["loss"]}.items()}


def _same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_other_stream_and_graphs(L):
    """The same bits eagerly, on a side stream, and from two captured graphs replayed on two streams at once."""
    one, two = Step(L, seed=1), Step(L, seed=2)
    want = []
    for st in (one, two):
        st.run()
        want.append(_snapshot(st))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one.run()
    side.synchronize()
    _same(_snapshot(one), want[0])
    graphs = []
    for st in (one, two):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            st.run()        # warm-up of the library's and of cuBLAS's state on this stream
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            st.run()
        graphs.append((g, s))
    for st in (one, two):
        for v in st.grads().values():
            v.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    _same(_snapshot(one), want[0])
    _same(_snapshot(two), want[1])


def test_kernels_wait_for_what_they_read(L):
    """Each call right behind the kernel that writes its inputs, behind work of another stream that was joined in, and behind
    a long kernel: eager, and replayed from a graph with such forks, where every kernel is set up ahead of its predecessor's end."""
    T, H, V = 512, 1024, 2000
    src = [torch.randn(T, H, device="cuda").to(BF) for _ in range(4)]
    W = (torch.randn(V, H, device="cuda") * H ** -0.5).to(BF)
    w = torch.ones(H, device="cuda", dtype=BF)
    lab = torch.randint(0, V, (T,), device="cuda")
    old, adv = torch.full((T,), -8.0, device="cuda"), torch.ones(1, device="cuda")
    big = torch.empty(1 << 27, device="cuda")
    side = torch.cuda.Stream()
    ws_p = torch.empty(L.liger_linear_policy_workspace(T, H, V), dtype=torch.uint8, device="cuda")
    ws_l = torch.empty(L.liger_linear_logp_workspace(T, H, V), dtype=torch.uint8, device="cuda")
    ws_n = torch.empty(L.liger_block_norm_bwd_workspace(T, H, 0), dtype=torch.uint8, device="cuda")
    t = {k: torch.empty(T, H, device="cuda", dtype=BF) for k in ("z", "r", "h", "y", "s", "dg", "du", "dr", "dz", "dX")}
    t.update(dW=torch.empty_like(W), dwn=torch.empty_like(w), rh=torch.empty(T, device="cuda"), loss=torch.empty(1, device="cuda"),
             logp=torch.empty(T, device="cuda"))
    kept = (*L.liger_ckpt8_empty(T, H), *L.liger_ckpt8_empty(T, H))

    def run():
        for k in t:
            t[k].fill_(float("nan"))
        big.fill_(1.0)                                       # a long kernel, then short ones
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            big[:1 << 26].mul_(0.5)
            t["r"].copy_(src[1])
        t["z"].copy_(src[0])
        main.wait_stream(side)                               # joined: r comes from the other stream
        L.liger_block_norm_fwd(t["z"], t["r"], t["h"], t["y"], w_pre=w, rstd_h=t["rh"])
        L.liger_swiglu_fwd_ckpt8(t["h"], t["y"], t["s"], *kept)
        L.liger_swiglu_bwd_ckpt8(t["s"], *kept, t["dg"], t["du"])
        L.liger_linear_logp_fwd(t["s"], W, lab, t["logp"], ws_l, wait=False)
        L.liger_linear_policy_fwd_bwd(t["s"], W, lab, old, adv, t["loss"], t["dX"], t["dW"], ws_p, wait=False)
        L.liger_block_norm_bwd(t["dg"], t["dX"], None, t["h"], t["dr"], t["dz"], ws_n, w_pre=w, rstd_h=t["rh"], dw_pre=t["dwn"])
        big.fill_(2.0)

    def result():
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in t.items()}
    run()
    first = result()
    assert all(bool(torch.isfinite(v).all()) for v in first.values())
    h = (src[0].double() + src[1].double())
    assert bool(((first["h"].double() - h).abs() <= 2.0 ** -8 * h.abs()).all())   # the joined stream's r was read
    for _ in range(20):
        run()
    _same(result(), first)
    own = torch.cuda.Stream()
    own.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(own):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=own):
            run()
    for _ in range(20):
        g.replay()
    _same(result(), first)


def test_threads(L):
    """Steps of four threads at once, each on its own stream and buffers."""
    steps = [Step(L, seed=10 + i) for i in range(4)]
    want = []
    for st in steps:
        st.run(wait=True)
        want.append(_snapshot(st))
    torch.cuda.synchronize()
    errors = []

    def work(st):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    st.run(wait=True)
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=work, args=(st,)) for st in steps]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    for st, w in zip(steps, want):
        _same(_snapshot(st), w)


def test_block_norms_past_32_bits(L):
    """2.2e9 elements: rows at both ends and around the 2^31-th element against 64 bits."""
    rows, cols = 540000, 4096
    z, r, h, y = (torch.empty(rows, cols, device="cuda", dtype=BF) for _ in range(4))
    for t in (z, r):
        t.normal_()
    w = torch.rand(cols, device="cuda").to(BF) + 0.5
    rz, rh = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    L.liger_block_norm_fwd(z, r, h, y, w, w, w, rz, rh, eps=EPS)
    at = torch.tensor([0, 1, 524286, 524287, 524288, 524289, rows - 2, rows - 1], device="cuda")

    def ref(at):
        a, b, ww = z[at].double(), r[at].double(), w.double()
        hh = b + a * (a.square().mean(1, keepdim=True) + EPS).rsqrt() * ww * ww
        return hh, hh * (hh.square().mean(1, keepdim=True) + EPS).rsqrt() * ww
    hh, yy = ref(at)
    for got, want in ((h[at], hh), (y[at], yy)):
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
    ws = torch.empty(L.liger_block_norm_bwd_workspace(rows, cols, 1), dtype=torch.uint8, device="cuda")
    dr, dz = torch.empty_like(z), torch.empty_like(z)
    g = [torch.empty_like(w) for _ in range(3)]
    L.liger_block_norm_bwd(r, y, z, h, dr, dz, ws, w, w, w, rz, rh, *g)
    # the documented formulas, from the row scales as the forward wrote them (rstd_h is that of the unrounded h)
    H, Z, ww, sh, sz = h[at].double(), z[at].double(), w.double(), rh[at, None].double(), rz[at, None].double()
    u = y[at].double() * ww
    D = r[at].double() + sh * u - sh ** 3 / cols * (u * H).sum(1, keepdim=True) * H
    q = ww * ww
    dzz = sz * q * D - sz ** 3 / cols * (q * D * Z).sum(1, keepdim=True) * Z
    # |terms| stay below 40, their sums below 4096 times that over cols: 4096 / 32 + 60 roundings of 2^-24
    for got, want in ((dr[at], D), (dz[at], dzz)):
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 190 * 2.0 ** -24 * 40).all())


def test_tensors_of_another_device_are_refused(L):
    """What is not on the current device is not passed to the library."""
    x = torch.randn(4, 64).to(BF)
    c = x.cuda()
    q, s = L.liger_ckpt8_empty(4, 64)
    for call in (lambda: L.liger_block_norm_fwd(c, x, c, None), lambda: L.liger_swiglu_fwd_ckpt8(c, c, x, q, s, q, s),
                 lambda: L.liger_swiglu_bwd_ckpt8(c, q.cpu(), s, q, s, c, c),
                 lambda: L.liger_linear_logp_fwd(c, c, torch.zeros(4, dtype=torch.int64), torch.empty(4, device="cuda"), c)):
        with pytest.raises(ValueError):
            call()
