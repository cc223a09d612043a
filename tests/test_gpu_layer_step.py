"""The layer-norm layer's operators and scored logits as they are used: a layer with its head, forward and backward, in a row; eager
and captured calls, other streams, several threads, offsets past 2^31, the same bits from run to run."""
import math
import threading

import pytest
import torch

from layer_util import IGNORE, frequencies, gen, randn, rotate, scores

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
YARN = dict(theta=1e4, scaling="yarn", factor=8.0, low=1.0, high=32.0, orig_len=64.0)


def _code(dt):
    import transformer_rmsnorm_fwd_gb300 as L
    return L.LIGER_BF16 if dt is BF else L.LIGER_F32


class Layer:
    """norm - packed projection - rotation - attention (plain torch) - projection + residual - norm - MLP + residual - norm - head
    - scores, with the gradients of everything, from the framework's operators; the same from autograd in 64 bits."""

    def __init__(self, B, S, heads, D, rotary, inter, vocab, dtype, seed=0):
        g = gen(seed)
        self.B, self.S, self.n, self.D, self.R, self.dt = B, S, heads, D, rotary, dtype
        H = heads * D
        self.H, T = H, B * S
        w = lambda n, k: randn(g, n, k, std=1 / math.sqrt(k), dtype=dtype)      # noqa: E731
        v = lambda n, m=0.0: randn(g, n, std=0.1, mean=m, dtype=dtype)          # noqa: E731
        self.p = dict(n1=v(H, 1.0), c1=v(H), wqkv=w(3 * H, H), bqkv=v(3 * H), wo=w(H, H), bo=v(H), n2=v(H, 1.0), c2=v(H), wu=w(inter, H),
                      bu=v(inter), wd=w(H, inter), bd=v(H), n3=v(H, 1.0), c3=v(H), head=w(vocab, H))
        self.x = randn(g, T, H, dtype=dtype)
        self.y = torch.randint(0, vocab, (T,), device="cuda", generator=g)
        self.y[::5] = IGNORE
        self.ga, self.gh = randn(g, T), randn(g, T, std=0.1)
        self.causal = torch.full((S, S), float("-inf"), device="cuda").triu(1)

    def _attention(self, q, k, v):      # [B, S, n, D]
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
        a = torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(self.D) + self.causal.to(q.dtype), -1)
        return (a @ v).transpose(1, 2).reshape(self.B * self.S, self.H)

    def own(self):
        import transformer_rmsnorm_fwd_gb300 as L
        p, dt, T, H = self.p, self.dt, self.B * self.S, self.H
        V, inter = p["head"].shape[0], p["wu"].shape[0]
        e = lambda *s: torch.empty(*s, dtype=dt, device="cuda")     # noqa: E731
        f = lambda *s: torch.empty(*s, device="cuda")               # noqa: E731
        kept = torch.float16 if dt is BF else F32
        need = max(L.liger_layernorm_bwd_workspace(T, H), *(L.liger_linear_act_bwd_workspace(T, k, n, a, _code(dt)) for k, n, a in (
            (H, 3 * H, "none"), (H, H, "none"), (H, inter, "gelu_tanh"), (inter, H, "none"), (H, V, "none"))), 256)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")    # one workspace for every call, as they run one after the other
        m = [(f(T), f(T)) for _ in range(3)]
        # forward
        a1 = L.liger_layernorm_fwd(self.x, p["n1"], p["c1"], e(T, H), *m[0])
        qkv = L.liger_linear_act_fwd(a1, p["wqkv"], e(T, 3 * H), bias=p["bqkv"]).view(self.B, self.S, 3 * self.n, self.D)
        q, k, v = qkv[:, :, :self.n], qkv[:, :, self.n:2 * self.n], qkv[:, :, 2 * self.n:]
        qr, kr = (e(self.B, self.S, self.n, self.D) for _ in range(2))
        L.liger_rope_scaled_fwd(q, k, qr, kr, self.R, **YARN)
        at = [t.float().detach().requires_grad_() for t in (qr, kr, v)]
        o = self._attention(*at)
        ob = o.detach().to(dt)
        h1 = self.x.clone()
        L.liger_linear_act_fwd(ob, p["wo"], h1, bias=p["bo"], residual=h1)
        a2 = L.liger_layernorm_fwd(h1, p["n2"], p["c2"], e(T, H), *m[1])
        pre = torch.empty(T, inter, dtype=kept, device="cuda")
        u = L.liger_linear_act_fwd(a2, p["wu"], e(T, inter), bias=p["bu"], act="gelu_tanh", pre=pre)
        h2 = L.liger_linear_act_fwd(u, p["wd"], e(T, H), bias=p["bd"], residual=h1)
        a3 = L.liger_layernorm_fwd(h2, p["n3"], p["c3"], e(T, H), *m[2])
        z = L.liger_linear_act_fwd(a3, p["head"], e(T, V))
        s = dict(logp=f(T), row_max=f(T), log_sum=f(T), entropy=f(T), top_logp=f(T, 3), top_ids=torch.empty(T, 3, dtype=torch.int64, device="cuda"))
        L.liger_token_logp_fwd(z, self.y, s["logp"], s["row_max"], s["log_sum"], s["entropy"], s["top_logp"], s["top_ids"], temperature=0.9)
        out = dict(s, z=z)
        # backward; the logits' gradient takes the logits' place
        out["z"] = z.clone()
        L.liger_token_logp_bwd(z, self.y, s["row_max"], s["log_sum"], self.ga, z, s["entropy"], self.gh, temperature=0.9)
        d = {}

        def lin(dY, X, w, b=None, pre=None, act="none"):
            dX, d[w] = torch.empty_like(X), torch.empty_like(p[w])
            d[b or w + "_"] = torch.empty_like(p[b]) if b else None
            L.liger_linear_act_bwd(dY, X, p[w], dX, d[w], d[b or w + "_"], ws, pre=pre, act=act)
            return dX

        def norm(dy, x, n, c, stat, dres):
            dx, d[n], d[c] = torch.empty_like(x), torch.empty_like(p[n]), torch.empty_like(p[c])
            L.liger_layernorm_bwd(dy, x, p[n], *stat, dx, d[n], d[c], ws, dres=dres)
            return dx

        dh2 = norm(lin(z, a3, "head"), h2, "n3", "c3", m[2], None)
        du = lin(dh2, u, "wd", "bd")
        dh1 = norm(lin(du, a2, "wu", "bu", pre, "gelu_tanh"), h1, "n2", "c2", m[1], dh2)
        do = lin(dh1, ob, "wo", "bo")
        o.backward(do.float())
        dq, dk, dv = (t.grad.to(dt) for t in at)
        dqkv = e(self.B, self.S, 3 * self.n, self.D)
        dqkv[:, :, 2 * self.n:] = dv
        L.liger_rope_scaled_bwd(dq, dk, dqkv[:, :, :self.n], dqkv[:, :, self.n:2 * self.n], self.R, **YARN)
        d["x"] = norm(lin(dqkv.view(T, 3 * H), a1, "wqkv", "bqkv"), self.x, "n1", "c1", m[0], dh1)
        out["grads"] = {k: t for k, t in d.items() if t is not None}
        return out

    def reference(self):
        p = {k: t.double().requires_grad_() for k, t in self.p.items()}
        x = self.x.double().requires_grad_()
        norm = lambda t, w, b: torch.nn.functional.layer_norm(t, (self.H,), w, b, 1e-5)     # noqa: E731
        f, mul = frequencies(self.R, **YARN)
        pos = torch.arange(self.S, device="cuda").expand(self.B, self.S)
        qkv = (norm(x, p["n1"], p["c1"]) @ p["wqkv"].T + p["bqkv"]).view(self.B, self.S, 3 * self.n, self.D)
        q, k = (rotate(t, pos, f, mul, self.R, "half")[0] for t in (qkv[:, :, :self.n], qkv[:, :, self.n:2 * self.n]))
        h1 = x + self._attention(q, k, qkv[:, :, 2 * self.n:]) @ p["wo"].T + p["bo"]
        u = torch.nn.functional.gelu(norm(h1, p["n2"], p["c2"]) @ p["wu"].T + p["bu"], approximate="tanh")
        h2 = h1 + u @ p["wd"].T + p["bd"]
        z = norm(h2, p["n3"], p["c3"]) @ p["head"].T
        logp, m, ls, ent, _, _ = scores(z, self.y, 0.9, 3)
        ((logp * self.ga.double()).sum() + (ent * self.gh.double()).sum()).backward()
        grads = {k: t.grad for k, t in p.items()}
        return dict(z=z.detach(), logp=logp.detach(), entropy=ent.detach(), grads=dict(grads, x=x.grad))


# Relative errors in norm. One operator's are within 1e-5 in fp32 and, its output rounded to bf16, half a step (2^-9 in norm,
# 2^-8 at most); some twenty of them follow each other, and what one rounds the next hands on.
STEP_TOL = {F32: 2e-4, BF: 20 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,S,heads,D,rotary,inter,vocab", [(2, 40, 4, 32, 16, 384, 520), (1, 300, 4, 64, 64, 512, 1000), (3, 7, 2, 40, 20, 136, 264)])
def test_layer_and_head_in_a_row(cuda_lib, dtype, B, S, heads, D, rotary, inter, vocab):
    layer = Layer(B, S, heads, D, rotary, inter, vocab, dtype)
    got, ref = layer.own(), layer.reference()
    off = lambda a, b: float((a.double() - b).norm() / b.norm())        # noqa: E731
    for k in ("z", "logp", "entropy"):
        assert off(got[k], ref[k]) < STEP_TOL[dtype], k
    for k, t in ref["grads"].items():
        assert off(got["grads"][k], t) < STEP_TOL[dtype], k
    # the alternatives are those of the logits that the head gave
    assert torch.equal(got["top_ids"], scores(got["z"], layer.y, 0.9, 3)[5])


def _calls(dtype, seed=0):
    """One call of every operator, on tensors of its own: [(name, call, outputs)], forms of few and of many rows."""
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(seed)
    kept = torch.float16 if dtype is BF else F32
    calls = []

    def add(name, fn, *outs):
        calls.append((name, fn, [o for o in outs if o is not None]))

    for rows, cols in ((3, 512), (900, 512), (70, 333), (5, 30000)):
        x, dy, w, b = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype), randn(g, cols, dtype=dtype), randn(g, cols, dtype=dtype)
        y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        mu, rs = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ws = torch.empty(L.liger_layernorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")

        def norm(x=x, dy=dy, w=w, b=b, y=y, dx=dx, dw=dw, db=db, mu=mu, rs=rs, ws=ws):
            L.liger_layernorm_fwd(x, w, b, y, mu, rs)
            L.liger_layernorm_bwd(dy, x, w, mu, rs, dx, dw, db, ws)
        add(f"norm {rows} {cols}", norm, y, dx, dw, db, mu, rs)
    for T, H, N in ((2, 256, 512), (200, 320, 264), (2500, 128, 1024), (3000, 256, 2048), (9, 33, 41)):
        X, W, bias, R = randn(g, T, H, dtype=dtype), randn(g, N, H, std=0.05, dtype=dtype), randn(g, N, dtype=dtype), randn(g, T, N, dtype=dtype)
        dY, Y, pre = randn(g, T, N, dtype=dtype), torch.empty_like(R), torch.empty(T, N, dtype=kept, device="cuda")
        dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty_like(bias)
        ws = torch.empty(max(256, L.liger_linear_act_bwd_workspace(T, H, N, "silu", _code(dtype))), dtype=torch.uint8, device="cuda")

        def lin(X=X, W=W, bias=bias, R=R, dY=dY, Y=Y, pre=pre, dX=dX, dW=dW, db=db, ws=ws):
            L.liger_linear_act_fwd(X, W, Y, bias=bias, residual=R, act="silu", pre=pre)
            L.liger_linear_act_bwd(dY, X, W, dX, dW, db, ws, pre=pre, act="silu")
        add(f"linear {T} {H} {N}", lin, Y, pre, dX, dW, db)
    for B, S, D, R in ((4, 1, 64, 32), (2, 400, 64, 32), (1, 33, 20, 10)):
        q, k = randn(g, B, S, 6, D, dtype=dtype), randn(g, B, S, 2, D, dtype=dtype)
        a = [torch.empty_like(t) for t in (q, k, q, k)]

        def rope(q=q, k=k, a=a, R=R):
            L.liger_rope_scaled_fwd(q, k, a[0], a[1], R, **YARN)
            L.liger_rope_scaled_bwd(q, k, a[2], a[3], R, **YARN)
        add(f"rope {B} {S} {D}", rope, *a)
    for T, V in ((1, 50000), (700, 1001), (40, 20000)):
        z, t = randn(g, T, V, std=2.0, dtype=dtype), torch.randint(0, V, (T,), device="cuda", generator=g)
        o = [torch.empty(T, device="cuda") for _ in range(4)]
        tl, ti, dz, gr = torch.empty(T, 5, device="cuda"), torch.empty(T, 5, dtype=torch.int64, device="cuda"), torch.empty_like(z), randn(g, T)

        def score(z=z, t=t, o=o, tl=tl, ti=ti, dz=dz, gr=gr):
            L.liger_token_logp_fwd(z, t, o[0], row_max=o[1], log_sum=o[2], entropy=o[3], top_logp=tl, top_ids=ti)
            L.liger_token_logp_bwd(z, t, o[1], o[2], gr, dz, entropy=o[3], g_entropy=gr)
        add(f"score {T} {V}", score, *o, tl, ti, dz)
    return calls


def _spoil(outs):
    for o in outs:
        o.fill_(77)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_calls_and_the_same_bits_again(cuda_lib, dtype):
    """Eager twice, captured alone and all in one graph, replayed twice: the same bits each time."""
    calls = _calls(dtype)
    want = {}
    for name, fn, outs in calls:
        fn()
        want[name] = [o.clone() for o in outs]
    for name, fn, outs in calls:
        _spoil(outs)
        fn()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    whole, single = torch.cuda.CUDAGraph(), []
    with torch.cuda.stream(stream):
        with torch.cuda.graph(whole, stream=stream):
            for _, fn, _ in calls:
                fn()
        for name, fn, outs in calls[::3]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                fn()
            single.append((name, g, outs))
    torch.cuda.synchronize()
    for _ in range(2):
        for _, _, outs in calls:
            _spoil(outs)
        whole.replay()
        for name, _, outs in calls:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name
    for name, g, outs in single:
        _spoil(outs)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name


def test_another_stream_waits_for_its_inputs(cuda_lib):
    """Calls on a side stream behind the kernels that write their inputs, which are the current stream's tensors."""
    import transformer_rmsnorm_fwd_gb300 as L
    side = torch.cuda.Stream()
    src = randn(gen(1), 4096, 2048, dtype=BF)
    W = randn(gen(2), 2048, 2048, std=0.02, dtype=BF)
    ref = L.liger_linear_act_fwd(L.liger_layernorm_fwd(src, None, None, torch.empty_like(src)), W, torch.empty_like(src), act="relu")
    torch.cuda.synchronize()
    for _ in range(5):
        x, a, y = torch.zeros_like(src), torch.zeros_like(src), torch.zeros_like(src)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                x.mul_(0.5)
            x.copy_(src)
            L.liger_layernorm_fwd(x, None, None, a)
            L.liger_linear_act_fwd(a, W, y, act="relu")
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, ref)


def test_several_threads(cuda_lib):
    """The same calls from four host threads at once, on tensors, workspaces and streams of their own."""
    sets = [_calls(BF, seed) for seed in range(4)]
    want = []
    for calls in sets:
        for _, fn, _ in calls:
            fn()
        want.append([[o.clone() for o in outs] for _, _, outs in calls])
    torch.cuda.synchronize()
    errors = []

    def work(calls):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    for _, fn, outs in calls:
                        _spoil(outs)
                        fn()
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for calls, w in zip(sets, want):
        for (name, _, outs), ref in zip(calls, w):
            assert all(torch.equal(a, b) for a, b in zip(outs, ref)), name


def test_offsets_past_32_bits(cuda_lib):
    """Tensors of more than 2^31 elements: the last rows come out as they do alone."""
    import transformer_rmsnorm_fwd_gb300 as L
    # logits: 17000 rows of 131072
    T, V = 17000, 131072
    z = torch.zeros(T, V, dtype=BF, device="cuda")
    z[-3:] = randn(gen(0), 3, V, std=2.0, dtype=BF)
    y = torch.randint(0, V, (T,), device="cuda", generator=gen(1))
    o = [torch.empty(T, device="cuda") for _ in range(4)]
    tl, ti = torch.empty(T, 4, device="cuda"), torch.empty(T, 4, dtype=torch.int64, device="cuda")
    L.liger_token_logp_fwd(z, y, o[0], row_max=o[1], log_sum=o[2], entropy=o[3], top_logp=tl, top_ids=ti)
    last = [torch.empty(3, device="cuda") for _ in range(4)]
    tl3, ti3 = torch.empty(3, 4, device="cuda"), torch.empty(3, 4, dtype=torch.int64, device="cuda")
    L.liger_token_logp_fwd(z[-3:], y[-3:], last[0], row_max=last[1], log_sum=last[2], entropy=last[3], top_logp=tl3, top_ids=ti3)
    assert torch.equal(ti[-3:], ti3)
    for a, b in zip(o, last):       # (a few rows are split over clusters of blocks: other groupings of the same sums)
        assert float((a[-3:] - b).abs().max()) < 1e-4
    # (its gradient is formed element by element: the same bits)
    few, cut = torch.empty(3, V, dtype=BF, device="cuda"), [t[-3:].clone() for t in (z, y, o[1], o[2], o[3])]
    L.liger_token_logp_bwd(*cut, few)
    L.liger_token_logp_bwd(z, y, o[1], o[2], o[3], z)
    assert torch.equal(z[-3:], few) and bool(few.any())
    del z
    # rows of a norm, in place
    x = torch.zeros((1 << 31) // 4096 + 40, 4096, dtype=BF, device="cuda")
    x[-2:] = randn(gen(2), 2, 4096, dtype=BF)
    ref = L.liger_layernorm_fwd(x[-2:].clone(), None, None, torch.empty_like(x[-2:]))
    L.liger_layernorm_fwd(x, None, None, x)
    assert torch.equal(x[-2:], ref) and not x[:5].any()
    del x
    # a projection's output, and the gradients back from it
    T, H, N = 200100, 64, 11008
    X, W = torch.zeros(T, H, dtype=BF, device="cuda"), randn(gen(3), N, H, dtype=BF)
    X[-300:] = randn(gen(4), 300, H, dtype=BF)
    Y, pre = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, N, dtype=torch.float16, device="cuda")
    L.liger_linear_act_fwd(X, W, Y, act="gelu", pre=pre)
    p = X[-300:].double() @ W.double().T
    assert float((Y[-300:].double() - torch.nn.functional.gelu(p)).norm() / p.norm()) < 2.0 ** -8 and not Y[:100].any()
    Y[:-300] = 0
    ws = torch.empty(L.liger_linear_act_bwd_workspace(T, H, N, "gelu"), dtype=torch.uint8, device="cuda")
    dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty(N, dtype=BF, device="cuda")
    L.liger_linear_act_bwd(Y, X, W, dX, dW, db, ws, pre=pre, act="gelu")
    q = pre[-300:].double().requires_grad_()
    torch.nn.functional.gelu(q).backward(Y[-300:].double())
    for got, want in ((dX[-300:], q.grad @ W.double()), (dW, q.grad.T @ X[-300:].double()), (db, q.grad.sum(0))):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -7
    assert not dX[:100].any()
    del X, Y, pre, ws, dX, dW
    # token rows of a rotation
    B, S, n, D = 1, 420000, 80, 64
    q = torch.zeros(B, S, n, D, dtype=BF, device="cuda")
    q[:, -2:] = randn(gen(5), 1, 2, n, D, dtype=BF)
    pos = torch.arange(S, device="cuda", dtype=torch.int32)[None].contiguous()
    few = torch.empty(1, 2, n, D, dtype=BF, device="cuda")
    L.liger_rope_scaled_fwd(q[:, -2:], None, few, None, 32, pos=pos[:, -2:].contiguous(), **YARN)
    L.liger_rope_scaled_fwd(q, None, q, None, 32, **YARN)
    assert torch.equal(q[:, -2:], few) and not q[:, :3].any()


def test_no_wait_has_expired(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    for _, fn, _ in _calls(BF, 9):
        fn()
    L.liger_device_status()
