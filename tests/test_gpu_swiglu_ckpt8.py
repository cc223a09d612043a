"""SwiGLU with 8-bit checkpoints, elementwise and in FusedLinearSwiGLU, against the definition in 64 bits: the codes and
scale bytes bit for bit, the activation and the gradients from the values read back."""
import pytest
import torch

from train_util import check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def L(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as lib
    return lib


def _pack(x):
    """Codes and scale bytes of x by the definition (64 bits; the step is a power of two, so nothing is rounded but the code)."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 32)).view(rows, -1, 32)
    bad = ~torch.isfinite(v).all(2)
    top = torch.where(bad[..., None], 0.0, v).abs().amax(2)
    _, e = torch.frexp(top)
    E = (e - 1).double()
    none = top < 2.0 ** -111
    step = torch.where(none, 1.0, torch.exp2(E - 6))
    codes = torch.where((none | bad)[..., None], 0.0, (torch.nan_to_num(v, 0, 0, 0) / step[..., None]).round().clamp(-127, 127))
    scale = torch.where(bad, 255.0, torch.where(none, 0.0, E + 127))
    return codes.view(rows, -1)[:, :cols].to(torch.int8), scale.to(torch.uint8), bad


def _read(codes, scale):
    cols = codes.shape[1]
    s = scale.double().repeat_interleave(32, 1)[:, :cols]
    step = torch.where(s == 0, 0.0, torch.exp2(s - 133))
    return torch.where(s == 255, float("nan"), codes.double() * step)


def _act64(g, u):
    return g * torch.sigmoid(g) * u


def _grads64(g, u, dy):
    s = torch.sigmoid(g)
    return dy * u * s * (1 + g * (1 - s)), dy * g * s


def _step(L, g, u, dy, in_place=False):
    rows, cols = g.shape
    g8, gs = L.liger_ckpt8_empty(rows, cols)
    u8, us = L.liger_ckpt8_empty(rows, cols)
    for t in (g8, gs, u8, us):
        t.fill_(77)
    y = g.clone() if in_place else torch.full_like(g, 7.0)
    L.liger_swiglu_fwd_ckpt8(y if in_place else g, u, y, g8, gs, u8, us)
    dg = dy.clone() if in_place else torch.full_like(g, 7.0)
    du = torch.full_like(g, 7.0)
    L.liger_swiglu_bwd_ckpt8(dg if in_place else dy, g8, gs, u8, us, dg, du)
    return y, (g8, gs), (u8, us), dg, du


# sigmoid in fp32: exp and the division add a few 2^-24 of their own size; for bf16 storage the fast
# exp and reciprocal are off by 2 ulp + |g| 2^-24 (exp's argument) and 2 ulp: chain of 16 + |g| over
# the terms' size covers both
def _chain(g):
    return 24 + 2 * g.abs()


def _check_step(L, g, u, dy, in_place=False):
    y, (g8, gs), (u8, us), dg, du = _step(L, g, u, dy, in_place)
    check(y, _act64(g.double(), u.double()), _act64(g.double(), u.double()).abs(), _chain(g.double()), "y")
    for codes, scale, x in ((g8, gs, g), (u8, us, u)):
        c64, s64, bad = _pack(x)
        assert torch.equal(scale, s64)
        keep = ~bad.repeat_interleave(32, 1)[:, :x.shape[1]]
        assert torch.equal(codes[keep], c64[keep])
        back = _read(codes, scale)
        step = torch.exp2(scale.double() - 133).repeat_interleave(32, 1)[:, :x.shape[1]]
        fine = keep & (scale.repeat_interleave(32, 1)[:, :x.shape[1]] > 0)
        off = (back - x.double()).abs()
        assert bool((off <= step)[fine].all())
        assert bool((off <= step / 2)[fine & (x.double().abs() <= 127.5 * step)].all())
    G, U = _read(g8, gs), _read(u8, us)
    rg, ru = _grads64(G, U, dy.double())
    d, s = dy.double().abs(), torch.sigmoid(G)
    # 1 + g (1 - s): its terms can cancel, so its error counts 1 + |g (1 - s)|
    check(dg, rg, d * U.abs() * s * (1 + (G * (1 - s)).abs() + G.abs()), _chain(torch.nan_to_num(G)), "dgate")
    check(du, ru, ru.abs(), _chain(torch.nan_to_num(G)), "dup")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (1, 32), (3, 31), (5, 33), (7, 40), (2, 688), (64, 1024), (129, 2739),
                                       (1000, 104), (17, 11008), (300, 520)])
def test_step(L, rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows * cols)
    g, u, dy = (torch.randn(rows, cols, device="cuda", generator=gen).to(DT[dtype]) * k for k in (2, 1, 1))
    _check_step(L, g, u, dy)
    _check_step(L, g, u, dy, in_place=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [96, 77])
def test_extreme_values(L, dtype, cols):
    """Groups of zeros, of tiny and of huge values, powers of two, codes at the rounding's halves and past 127.5 steps."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows = 40
    g = torch.randn(rows, cols, device="cuda", generator=gen)
    g[0] = 0
    g[1] = -0.0
    for r, e in enumerate(range(-126, 120, 8), start=2):
        g[r % rows] *= 2.0 ** e
    g[33] = torch.exp2(torch.arange(cols, device="cuda").float() % 9 - 4)
    g[34] = (torch.arange(cols, device="cuda").float() % 64 + 64.5) / 64          # halves of a step
    g[35] = 127.75 / 64
    g[36] = -255 / 128
    g[37] = 2.0 ** -111
    g[38] = 2.0 ** -112
    g = g.to(DT[dtype])
    u = torch.randn(rows, cols, device="cuda", generator=gen).to(DT[dtype])
    dy = torch.randn(rows, cols, device="cuda", generator=gen).to(DT[dtype])
    y, (g8, gs), _, dg, du = _step(L, g, u, dy)
    c64, s64, _ = _pack(g)
    assert torch.equal(gs, s64) and torch.equal(g8, c64)
    assert bool(torch.isfinite(dg.double()[3:]).any())
    _check_step(L, u, g.clamp(-2.0 ** 40, 2.0 ** 40), dy)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [128, 67])
def test_infinities_stay_in_their_group(L, dtype, cols):
    gen = torch.Generator(device="cuda").manual_seed(6)
    g, u, dy = (torch.randn(4, cols, device="cuda", generator=gen).to(DT[dtype]) for _ in range(3))
    g[1, 5], u[2, 40], g[3, 33] = float("nan"), float("inf"), float("-inf")
    _, (g8, gs), (u8, us), dg, du = _step(L, g, u, dy)
    for codes, scale, x in ((g8, gs, g), (u8, us, u)):
        c64, s64, bad = _pack(x)
        assert torch.equal(scale, s64)
        keep = ~bad.repeat_interleave(32, 1)[:, :cols]
        assert torch.equal(codes[keep], c64[keep])
    G, U = _read(g8, gs), _read(u8, us)
    hit = torch.isnan(G) | torch.isnan(U)
    assert int(hit.sum()) == 3 * 32 and torch.equal(torch.isnan(dg), hit) and torch.equal(torch.isnan(du), torch.isnan(G))


def test_empty(L):
    e = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    q, s = L.liger_ckpt8_empty(0, 64)
    L.liger_swiglu_fwd_ckpt8(e, e, e, q, s, q, s)
    L.liger_swiglu_bwd_ckpt8(e, q, s, q, s, e, e)


def test_past_32_bits(L):
    """Offsets beyond 2^31 elements: the last rows of a tall tensor equal those of a short one."""
    rows, cols = 16640, 131072      # 2.18e9 elements
    tail = torch.randn(2, cols, device="cuda").to(torch.bfloat16)
    g = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    g[-2:] = tail
    q, s = L.liger_ckpt8_empty(rows, cols)
    L.liger_swiglu_fwd_ckpt8(g, g, g, q, s, q, s)
    one = torch.empty_like(tail)
    q1, s1 = L.liger_ckpt8_empty(2, cols)
    L.liger_swiglu_fwd_ckpt8(tail, tail, one, q1, s1, q1, s1)
    assert torch.equal(g[-2:], one) and torch.equal(q[-2:], q1) and torch.equal(s[-2:], s1)
    assert bool((g[:-2].view(torch.int16).amax() == 0))
    L.liger_swiglu_bwd_ckpt8(g, q, s, q, s, g, g.clone())


def _linear_inputs(T, H, I, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf = torch.bfloat16
    X, dH = torch.randn(T, H, device="cuda", generator=gen).to(bf), torch.randn(T, I, device="cuda", generator=gen).to(bf)
    Wg, Wu = ((torch.randn(I, H, device="cuda", generator=gen) * 1.3 * H ** -0.5).to(bf) for _ in range(2))
    return X, Wg, Wu, dH


@pytest.mark.parametrize("T,H,I", [(1, 64, 8), (3, 72, 40), (130, 128, 136), (257, 520, 696), (300, 1024, 256), (64, 64, 1376),
                                   (5000, 256, 320),
                                   # dX split along K over idle CTA pairs: one row, part of a row tile, several
                                   # column tiles, k ranges that do not divide the k-blocks
                                   (1, 112, 9016), (7, 520, 2056), (200, 264, 8200), (300, 72, 6000)])
def test_linear_step(L, T, H, I):
    X, Wg, Wu, dH = _linear_inputs(T, H, I, T)
    g8, gs = L.liger_ckpt8_empty(T, I)
    u8, us = L.liger_ckpt8_empty(T, I)
    for t in (g8, gs, u8, us):
        t.fill_(77)
    out = torch.full_like(dH, 7.0)
    L.liger_fused_linear_swiglu_fwd_ckpt8(X, Wg, Wu, out, g8, gs, u8, us)
    plain = torch.empty_like(out)
    L.liger_fused_linear_swiglu_fwd(X, Wg, Wu, plain)
    assert torch.equal(out, plain)
    x64, g64, u64 = X.double(), X.double() @ Wg.double().T, X.double() @ Wu.double().T
    # the fp32 products are off by at most H 2^-23 of the terms' sizes (tensor-core sums round toward
    # zero); a code may then fall to the other side of a half, one step away
    for codes, scale, z, W in ((g8, gs, g64, Wg), (u8, us, u64, Wu)):
        err = H * 2.0 ** -23 * (x64.abs() @ W.double().abs().T)
        c64, s64, _ = _pack(z)
        step = torch.exp2(scale.double() - 133).repeat_interleave(32, 1)[:, :I]
        top = torch.nn.functional.pad(z.abs(), (0, -I % 32)).view(T, -1, 32).amax(2)
        room = torch.nn.functional.pad(err, (0, -I % 32)).view(T, -1, 32).amax(2)
        moved = scale != s64                        # only where the largest value is next to a power of two
        lo, hi = torch.floor(torch.log2(top - room)), torch.floor(torch.log2(top + room))
        assert bool(((lo != hi) | ~moved).all())
        assert bool(((_read(codes, scale) - z).abs() <= step + err).all())
    G, U = _read(g8, gs), _read(u8, us)
    dg64, du64 = _grads64(G, U, dH.double())
    ws = torch.empty(max(L.liger_fused_linear_swiglu_workspace(T, I), 256), dtype=torch.uint8, device="cuda")
    dX, dWg, dWu = torch.full_like(X, 7.0), torch.full_like(Wg, 7.0), torch.full_like(Wu, 7.0)
    L.liger_fused_linear_swiglu_bwd_ckpt8(X, Wg, Wu, dH, g8, gs, u8, us, dX, dWg, dWu, ws)
    # dG and dU are rounded to bf16 (2^-8 of each term) before the products; fp32 sums over K
    bf = 2.0 ** 16      # one bf16 half step, 2^-8, in units of 2^-24
    mg = dg64.abs() @ Wg.double().abs() + du64.abs() @ Wu.double().abs()
    check(dX, dg64 @ Wg.double() + du64 @ Wu.double(), mg, bf + 4 * I + 100, "dX")
    check(dWg, dg64.T @ x64, dg64.abs().T @ x64.abs(), bf + 2 * T + 100, "dWg")
    check(dWu, du64.T @ x64, du64.abs().T @ x64.abs(), bf + 2 * T + 100, "dWu")


@pytest.mark.parametrize("T,H,I", [(4100, 1032, 2040), (4096, 264, 5000), (8200, 2056, 1104), (4351, 328, 5000)])
def test_linear_step_of_many_tokens(L, T, H, I):
    """The last round of dW's tiles split over the tokens (several column blocks, ragged row blocks of both weights, both tile
    orders), and a forward whose rows are swept in two groups (8200 x 2056)."""
    test_linear_step(L, T, H, I)


def test_linear_gradient_against_differences(L):
    """The backward of the checkpointed values is the slope of the plain MLP within what 8 bits allow: the directional
    derivative of sum(dH * out) along a change of Wu, whose gradient uses g read back (error <= 1/128 of a group's top)."""
    T, H, I = 200, 128, 64
    X, Wg, Wu, dH = _linear_inputs(T, H, I, 3)
    g8, gs = L.liger_ckpt8_empty(T, I)
    u8, us = L.liger_ckpt8_empty(T, I)
    out, ws = torch.empty_like(dH), torch.empty(L.liger_fused_linear_swiglu_workspace(T, I), dtype=torch.uint8, device="cuda")
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    L.liger_fused_linear_swiglu_fwd_ckpt8(X, Wg, Wu, out, g8, gs, u8, us)
    L.liger_fused_linear_swiglu_bwd_ckpt8(X, Wg, Wu, dH, g8, gs, u8, us, dX, dWg, dWu, ws)
    x, wg, wu, dh = X.double(), Wg.double(), Wu.double(), dH.double()
    v = torch.randn(I, H, device="cuda", dtype=torch.float64)

    def value(w):
        return float((_act64(x @ wg.T, x @ w.T) * dh).sum())
    slope = (value(wu + 1e-5 * v) - value(wu - 1e-5 * v)) / 2e-5
    # sum over t, i of dh silu'(..) (x v): g is off by at most top / 128 (half a step of top / 64 or less)
    # and |silu'| <= 1.1; bf16 roundings of dU and dWu: 2^-8 each
    xv = (x @ v.T).abs() * dh.abs()
    top = (x @ wg.T).abs().amax() / 64
    allowed = float((xv * (1.1 * top + 2 * 2.0 ** -8 * (x @ wg.T).abs())).sum())
    assert abs(float((dWu.double() * v).sum()) - slope) <= allowed


def test_linear_no_tokens(L):
    X, Wg, Wu, dH = _linear_inputs(0, 64, 32, 1)
    q, s = L.liger_ckpt8_empty(0, 32)
    L.liger_fused_linear_swiglu_fwd_ckpt8(X, Wg, Wu, torch.empty_like(dH), q, s, q, s)
    dWg, dWu = torch.full_like(Wg, 7.0), torch.full_like(Wu, 7.0)
    L.liger_fused_linear_swiglu_bwd_ckpt8(X, Wg, Wu, dH, q, s, q, s, torch.empty_like(X), dWg, dWu, None)
    assert bool((dWg == 0).all()) and bool((dWu == 0).all())


def test_refusals(L):
    g = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    q, s = L.liger_ckpt8_empty(4, 64)
    with pytest.raises(ValueError):
        L.liger_swiglu_fwd_ckpt8(g, g, g, q, s[:, :1].contiguous(), q, s)
    with pytest.raises(TypeError):
        L.liger_swiglu_fwd_ckpt8(g, g, g, q.to(torch.uint8), s, q, s)
    with pytest.raises(TypeError):
        L.liger_swiglu_bwd_ckpt8(g, q, s, q, s, g.float(), g)
    with pytest.raises(TypeError):
        L.liger_swiglu_fwd_ckpt8(g.half(), g.half(), g.half(), q, s, q, s)
    X, Wg, Wu, dH = _linear_inputs(4, 64, 64, 1)
    with pytest.raises(L.LigerError) as e:      # fp32: the tensor-core path is bf16
        L.liger_fused_linear_swiglu_fwd_ckpt8(X.float(), Wg.float(), Wu.float(), dH.float(), q, s, q, s)
    assert e.value.status == -3
    with pytest.raises(L.LigerError) as e:
        L.liger_fused_linear_swiglu_bwd_ckpt8(X, Wg, Wu, dH, q, s, q, s, X.clone(), Wg.clone(), Wu.clone(), None)
    assert e.value.status == -6
