"""Token log-probabilities, entropy and alternatives of logits against their formulas in 64 bits, and the gradient."""
import math

import pytest
import torch

from layer_util import IGNORE, gen, randn, scores
from train_util import check

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
NINF = float("-inf")


def _outputs(T, k):
    f = lambda *s: torch.full(s, 7.0, device="cuda")       # noqa: E731
    return dict(logp=f(T), row_max=f(T), log_sum=f(T), entropy=f(T), top_logp=f(T, k) if k else None,
                top_ids=torch.full((T, k), -7, dtype=torch.int64, device="cuda") if k else None)


def forward(z, tokens, k, temp=1.0):
    import transformer_rmsnorm_fwd_gb300 as L
    o = _outputs(z.shape[0], k)
    L.liger_token_logp_fwd(z, tokens, o["logp"], row_max=o["row_max"], log_sum=o["log_sum"], entropy=o["entropy"],
                           top_logp=o["top_logp"], top_ids=o["top_ids"], temperature=temp)
    return o


def _chain(V):
    # a sum of V terms (at most V / 128 in one register, then a tree), 2^d (2^-22 of it, and 2^-24 |d| of rounding in d: the
    # weights 2^d make that at most log2 V + 2 on average), the logarithm
    return V / 128 + 100


def compare(z, tokens, k, temp, o):
    logp, m, ls, ent, top, ids = scores(z, tokens, temp, k)
    c, one = _chain(z.shape[1]), torch.ones_like(ls)
    assert torch.equal(o["row_max"].double(), m)
    check(o["log_sum"], ls, one, c, "log_sum")
    check(o["logp"], logp, one + logp.abs(), c, "logp")
    check(o["entropy"], ent, one + 2 * ls, c, "entropy")
    if k:
        assert torch.equal(o["top_ids"], ids)
        check(o["top_logp"], top, 1 + top.abs(), c, "top_logp")


def tokens_of(g, T, V, ignored=True):
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    if ignored and T > 2:
        y[T // 2] = IGNORE
    return y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 2, 2), (5, 7, 7), (4, 32, 32), (9, 33, 20), (2, 255, 1), (40, 1000, 5), (7, 1001, 32),
                                   (33, 1024, 8), (11, 4096, 20), (600, 515, 3), (6, 8191, 10), (3, 32771, 20), (17, 50001, 8), (2, 128256, 20),
                                   (1, 151936, 32), (5, 151937, 1), (1, 300000, 20), (700, 9000, 4), (3, 128256, 0)])
def test_shapes(cuda_lib, dtype, T, V, k):
    g = gen(T + V)
    z = randn(g, T, V, std=2.5, dtype=dtype)
    y = tokens_of(g, T, V)
    compare(z, y, k, 1.0, forward(z, y, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,pad", [(1000, 8), (1000, 1), (4097, 3), (30000, 5), (64, 64)])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_strides_and_unaligned_rows(cuda_lib, dtype, V, pad, first):
    """Rows of a wider buffer, from any element on: what stands beside them is not read as a logit."""
    g = gen(V + pad)
    T = 6
    buf = torch.full((T, V + pad + first), 1e30, dtype=dtype, device="cuda")
    z = buf[:, first:first + V]
    z.copy_(randn(g, T, V, std=2.0, dtype=dtype))
    y = tokens_of(g, T, V)
    compare(z.contiguous(), y, 6, 0.7, forward(z, y, 6, 0.7))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("temp", [0.05, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("V", [100, 20000])
def test_temperatures_and_sizes(cuda_lib, dtype, temp, V):
    g = gen(3)
    for std, mean in ((0.01, 0.0), (3.0, 5000.0), (50.0, -100.0)):
        z = randn(g, 5, V, std=std, mean=mean, dtype=dtype)
        y = tokens_of(g, 5, V)
        a = ((z.double() - z.double().max(1, keepdim=True).values) / temp)
        logp, m, ls, ent, top, ids = scores(z, y, temp, 9)
        o = forward(z, y, 9, temp)
        p = torch.softmax(a, 1)
        # z - m and its quotient are rounded: relative to their size
        wide = 1 + 3 * (p * a.abs()).sum(1)
        c = _chain(V)
        check(o["log_sum"], ls, wide, c, "log_sum")
        check(o["entropy"], ent, wide * (1 + wide), c, "entropy")
        check(o["logp"], logp, wide + logp.abs(), c, "logp")
        check(o["top_logp"], top, wide[:, None] + top.abs(), c, "top_logp")
        assert torch.equal(o["top_ids"], ids)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [64, 1000, 40001])
def test_masks(cuda_lib, dtype, V):
    """-inf and the type's lowest value as masks; rows with one word left, and fewer words left than alternatives asked for."""
    g = gen(V)
    z = randn(g, 8, V, std=2.0, dtype=dtype)
    drop = torch.rand(8, V, device="cuda", generator=g) < 0.9
    z[:4] = torch.where(drop[:4], torch.tensor(NINF, dtype=dtype, device="cuda"), z[:4])
    z[4:] = torch.where(drop[4:], torch.tensor(torch.finfo(dtype).min, dtype=dtype, device="cuda"), z[4:])
    z[1] = NINF
    z[1, V // 3] = 1.5
    z[5] = torch.finfo(dtype).min
    z[5, V - 1] = -3.0
    z[6] = torch.finfo(dtype).min           # all of the row: uniform
    z[0, 0] = z[2, 0] = z[3, 0] = 0.5
    y = torch.tensor([0, V // 3, 0, 0, V // 2, V - 1, 3, 1], device="cuda")
    k = min(32, V)
    o = forward(z, y, k)
    logp, m, ls, ent, top, ids = scores(z, y, 1.0, k)
    c = _chain(V)
    check(o["log_sum"], ls, torch.ones_like(ls), c, "log_sum")
    check(o["entropy"], ent, 1 + 2 * ls, c, "entropy")
    assert torch.equal(o["top_ids"], ids)
    low = float(torch.finfo(dtype).min) / 2
    keep = logp > low                       # (differences of the lowest value lose nothing either, but may round to -inf)
    check(o["logp"][keep], logp[keep], 1 + logp[keep].abs(), c, "logp")
    live = top > low
    check(o["top_logp"][live], top[live], 1 + top[live].abs(), c, "top_logp")
    assert bool((o["top_logp"][~live].double() <= low).all())
    assert float(o["entropy"][1]) == 0 and float(o["logp"][1]) == 0 and float(o["logp"][5]) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [40, 5000, 131071])
def test_rows_without_a_word(cuda_lib, dtype, V):
    import transformer_rmsnorm_fwd_gb300 as L
    z = randn(gen(V), 3, V, dtype=dtype)
    z[1] = NINF
    y = torch.tensor([1, 2, 3], device="cuda")
    o = forward(z, y, 5)
    assert float(o["row_max"][1]) == float(o["log_sum"][1]) == float(o["logp"][1]) == NINF and float(o["entropy"][1]) == 0
    assert o["top_ids"][1].tolist() == [0, 1, 2, 3, 4] and bool((o["top_logp"][1] == NINF).all())
    sel = torch.tensor([0, 2], device="cuda")
    compare(z[sel], y[sel], 5, 1.0, {n: v[sel] for n, v in o.items()})
    d = torch.full_like(z, 7.0)
    one = torch.ones(3, device="cuda")
    L.liger_token_logp_bwd(z, y, o["row_max"], o["log_sum"], one, d, entropy=o["entropy"], g_entropy=one)
    assert not d[1].any() and bool(torch.isfinite(d).all()) and bool(d[0].any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [64, 3000, 128256])
@pytest.mark.parametrize("kind", ["constant", "two values", "ascending", "descending", "one block", "every 512th", "zeros of both signs"])
def test_ties_and_orders(cuda_lib, dtype, V, kind):
    """Equal logits go by their index, wherever in the row the largest stand."""
    i = torch.arange(V, device="cuda")
    if kind == "constant":
        row = torch.full((V,), 2.5, device="cuda")
    elif kind == "two values":
        row = (i * 7919 % 3 == 0).float()
    elif kind == "ascending":
        row = i.float() / V * 8
    elif kind == "descending":
        row = -i.float() / V * 8
    elif kind == "one block":                   # more equal largest ones side by side than alternatives
        row = ((i >= V // 2) & (i < V // 2 + 5000)).float() * 4
    elif kind == "every 512th":
        row = (i % 512 == 3).float() * 4 + (i % 4096 == 11).float() * (1 + i.float() / V)
    else:
        row = torch.where(i % 2 == 0, -0.0, 0.0)
    z = torch.stack([row, row.flip(0), -row]).to(dtype)
    y = torch.tensor([0, V - 1, IGNORE], device="cuda")
    for k in (1, 32):
        compare(z, y, k, 1.0, forward(z, y, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [50, 9001, 100000])
def test_nan_and_infinities_stay_in_their_rows(cuda_lib, dtype, V):
    z = randn(gen(V), 5, V, dtype=dtype)
    y = torch.tensor([0, 1, 2, V, -3], device="cuda")
    compare(z[:3], y[:3], 4, 1.0, {n: v[:3] for n, v in forward(z, y, 4).items()})
    assert bool(torch.isnan(forward(z, y, 4)["logp"][3:]).all())        # tokens outside the vocabulary
    z[1, V // 2], z[1, 7] = float("nan"), float("nan")
    z[2, 9] = float("inf")
    o = forward(z, y, 4)
    for n in ("log_sum", "entropy", "logp"):
        assert bool(torch.isnan(o[n][1:3]).all()), n
    assert bool(torch.isnan(o["top_logp"][1:3]).all())
    assert sorted([7, V // 2]) == o["top_ids"][1, :2].tolist() and int(o["top_ids"][2, 0]) == 9
    compare(z[:1], y[:1], 4, 1.0, {n: v[:1] for n, v in o.items()})


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k", [(300, 3), (2048, 8), (2100, 32), (20001, 5), (32771, 20)])
def test_many_rows(cuda_lib, dtype, V, k):
    """A batch large enough for fewer threads a row: against 64 bits, and odd rows against the same rows on their own."""
    T = 1000
    g = gen(V + k)
    z = randn(g, T, V, std=2.5, dtype=dtype)
    i = torch.arange(V, device="cuda")
    odd = torch.tensor([0, 5, 151, 152, 500, 608, 777, 911, T - 1], device="cuda")
    z[odd[0]] = 2.5                                     # all equal
    z[odd[1]] = (i * 7919 % 3 == 0).to(dtype)           # two values
    z[odd[2]] = NINF                                    # nothing left
    z[odd[3], 1:] = NINF                                # one word left
    z[odd[4]] = torch.where(i % 10 == 0, z[odd[4]], torch.tensor(torch.finfo(dtype).min, dtype=dtype, device="cuda"))
    z[odd[5], V // 2] = float("nan")
    z[odd[6], 9] = float("inf")
    z[odd[7]] = (i.float() / V * 8).to(dtype)           # ascending
    z[odd[8]] = ((i >= V // 2) & (i < V // 2 + 1500)).to(dtype) * 4
    y = tokens_of(g, T, V)
    y[odd[3]] = 0
    o, alone = forward(z, y, k), forward(z[odd], y[odd], k)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[odd] = False
    compare(z[rest], y[rest], k, 1.0, {n: v[rest] for n, v in o.items()})
    c = _chain(V)                                       # each of the two is within c
    for n, v in alone.items():
        u = o[n][odd]
        if n in ("top_ids", "row_max"):
            assert torch.equal(u.nan_to_num(nan=-5.0), v.nan_to_num(nan=-5.0)), n
            continue
        live = torch.isfinite(v)
        assert torch.equal(torch.isfinite(u), live) and torch.equal(torch.isnan(u), torch.isnan(v)), n
        check(u[live], v[live].double(), 2 + 2 * v[live].double().abs() + (2 * math.log(V) if n == "entropy" else 0), 2 * c, n)


def bwd_ref(z, y, m, ls, H, g, h, temp):
    """The gradient in 64 bits from the forward's fp32 outputs, and the magnitudes of its terms."""
    a = (z.double() - m.double()[:, None]) / temp - ls.double()[:, None]
    p = a.exp()
    a = torch.where(p > 0, a, torch.zeros_like(a))
    live = (y != IGNORE)
    g = torch.where(live, g.double(), torch.zeros_like(g.double()))[:, None] if g is not None else torch.zeros_like(a[:, :1])
    hot = torch.zeros_like(p)
    hot.scatter_(1, y.clamp(min=0)[:, None], live.double()[:, None])
    d, mag = g * (hot - p), g.abs() * (hot + p * (1 + a.abs()))
    if h is not None:
        h, H = h.double()[:, None], H.double()[:, None]
        d, mag = d - h * p * (a + H), mag + h.abs() * p * (a.abs() + H) * (1 + a.abs())
    return d / temp, mag / temp


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(1, 1), (2, 3), (5, 8), (9, 1001), (300, 515), (7, 4096), (3, 32771), (2, 151936)])
@pytest.mark.parametrize("parts", ["logp", "entropy", "both"])
def test_gradient(cuda_lib, dtype, T, V, parts):
    import transformer_rmsnorm_fwd_gb300 as L
    gn = gen(V)
    z = randn(gn, T, V, std=2.0, dtype=dtype)
    y = tokens_of(gn, T, V)
    temp = 0.8
    o = forward(z, y, 0, temp)
    g = randn(gn, T) if parts != "entropy" else None
    h = randn(gn, T) if parts != "logp" else None
    if g is not None:
        g[y == IGNORE] = float("nan")           # not read there
    d = torch.full_like(z, 7.0)
    L.liger_token_logp_bwd(z, y if g is not None else None, o["row_max"], o["log_sum"], g, d, entropy=o["entropy"] if h is not None else None,
                           g_entropy=h, temperature=temp)
    ref, mag = bwd_ref(z, y if g is not None else torch.full_like(y, IGNORE), o["row_max"], o["log_sum"], o["entropy"], g, h, temp)
    check(d, ref, mag, 16, "dlogits")
    same = z.clone()
    L.liger_token_logp_bwd(same, y if g is not None else None, o["row_max"], o["log_sum"], g, same,
                           entropy=o["entropy"] if h is not None else None, g_entropy=h, temperature=temp)
    assert torch.equal(same, d)
    if g is not None and h is None and T > 2:
        assert not d[y == IGNORE].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_strided_rows(cuda_lib, dtype):
    import transformer_rmsnorm_fwd_gb300 as L
    T, V = 5, 777
    gn = gen(1)
    buf = torch.full((T, V + 6), 3.0, dtype=dtype, device="cuda")
    out = torch.full((T, V + 11), 9.0, dtype=dtype, device="cuda")
    z, d = buf[:, 5:5 + V], out[:, 1:1 + V]
    z.copy_(randn(gn, T, V, std=2.0, dtype=dtype))
    z[2, 10:700] = NINF
    y = tokens_of(gn, T, V)
    g, h = randn(gn, T), randn(gn, T)
    o = forward(z, y, 0)
    L.liger_token_logp_bwd(z, y, o["row_max"], o["log_sum"], g, d, entropy=o["entropy"], g_entropy=h)
    ref, mag = bwd_ref(z, y, o["row_max"], o["log_sum"], o["entropy"], g, h, 1.0)
    check(d, ref, mag, 16, "dlogits")
    assert bool((out[:, :1] == 9).all()) and bool((out[:, 1 + V:] == 9).all())
    assert not d[2, 10:700].any()


def test_rows_without_a_gradient_are_zero_whatever_they_hold(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    z = randn(gen(0), 4, 300)
    z[0], z[2, 5] = float("nan"), float("inf")
    y = torch.tensor([IGNORE, 1, 2, 301], device="cuda")
    o = forward(z, y, 0)
    g, d = torch.tensor([1.0, 1.0, 0.0, 1.0], device="cuda"), torch.full_like(z, 7.0)
    L.liger_token_logp_bwd(z, y, o["row_max"], o["log_sum"], g, d)
    assert not d[0].any() and not d[2].any() and bool(torch.isfinite(d[1]).all())
    assert bool(torch.isnan(d[3]).any())        # a token outside the vocabulary


def test_gradient_against_differences(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    gn = gen(2)
    T, V, temp = 3, 12, 1.7
    z, y = randn(gn, T, V, std=1.5), torch.tensor([4, IGNORE, 11], device="cuda")
    g, h = randn(gn, T), randn(gn, T)
    o, d = forward(z, y, 0, temp), torch.empty_like(z)
    L.liger_token_logp_bwd(z, y, o["row_max"], o["log_sum"], g, d, entropy=o["entropy"], g_entropy=h, temperature=temp)

    def loss(v):
        logp, _, _, ent, _, _ = scores(v, y, temp, 1)
        return float((logp * g.double()).sum() + (ent * h.double()).sum())

    for i in range(z.numel()):
        up, down = z.double().clone(), z.double().clone()
        up.view(-1)[i] += 1e-5
        down.view(-1)[i] -= 1e-5
        assert abs((loss(up) - loss(down)) / 2e-5 - float(d.view(-1)[i])) < 2e-6, i


def test_optional_outputs(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    z, y = randn(gen(5), 6, 2000, dtype=torch.bfloat16), torch.arange(6, device="cuda")
    o = forward(z, y, 3)
    for only in o:
        a = {n: None for n in o}
        a[only] = torch.empty_like(o[only])
        if only.startswith("top"):
            a.update({n: torch.empty_like(o[n]) for n in ("top_ids", "top_logp")})
        L.liger_token_logp_fwd(z, y if only == "logp" else None, a["logp"], row_max=a["row_max"], log_sum=a["log_sum"],
                               entropy=a["entropy"], top_logp=a["top_logp"], top_ids=a["top_ids"])
        assert torch.equal(a[only], o[only]), only


def test_refusals(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    z, y, f = torch.zeros(4, 50, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.empty(4, device="cuda")
    for bad in (dict(tokens=y.int()), dict(tokens=y[:3]), dict(logp=f.double()), dict(logits=z.t()), dict(logits=z.half()),
                dict(logits=z[:, ::2]), dict(entropy=f[:2])):
        a = dict(dict(logits=z, tokens=y, logp=f, entropy=None), **bad)
        with pytest.raises((ValueError, TypeError)):
            L.liger_token_logp_fwd(a["logits"], a["tokens"], a["logp"], entropy=a["entropy"])
    ids, lp = torch.empty(4, 33, dtype=torch.int64, device="cuda"), torch.empty(4, 33, device="cuda")
    with pytest.raises(L.LigerError):
        L.liger_token_logp_fwd(z, y, f, top_logp=lp, top_ids=ids)
    with pytest.raises(L.LigerError):
        L.liger_token_logp_fwd(z, y, None)
    with pytest.raises(L.LigerError):
        L.liger_token_logp_fwd(z, y, f, temperature=0.0)
    with pytest.raises(L.LigerError):
        L.liger_token_logp_bwd(z, y, f, f, None, torch.empty_like(z))
