"""Layer norm against its formulas in 64 bits: types, widths, row counts, optional parts, aliases, rows far from 0."""
import pytest
import torch

from layer_util import gen, randn
from train_util import check

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _chain(cols):
    # sums over a row: at most cols / 32 terms in one register, then a tree and a few roundings of the result
    return cols / 32 + 40


def fwd_ref(x, w, b, eps):
    """y and the magnitudes of its terms, mean, rstd."""
    x = x.double()
    n = x.shape[-1]
    m = x.sum(1, keepdim=True) / n
    rs = 1 / torch.sqrt(((x - m) ** 2).sum(1, keepdim=True) / n + eps)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mag = (x.abs() + m.abs() + x.abs().sum(1, keepdim=True) / n) * rs * w.abs() + b.abs()
    return (x - m) * rs * w + b, mag, m[:, 0], rs[:, 0]


def bwd_ref(dy, dres, x, w, mean, rstd):
    dy, x, m, rs = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    xh, g = (x - m) * rs, dy * w
    dx = rs * (g - g.sum(1, keepdim=True) / n - xh * (g * xh).sum(1, keepdim=True) / n)
    mag = rs * (g.abs() + g.abs().sum(1, keepdim=True) / n + xh.abs() * (g * xh).abs().sum(1, keepdim=True) / n)
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    return dx, mag, (dy * xh).sum(0), (dy * xh).abs().sum(0), dy.sum(0), dy.abs().sum(0)


def run_case(lib, dtype, rows, cols, seed=0, weight=True, bias=True, residual=True, std=1.0, mean=0.3, eps=1e-5, x=None, in_place=""):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(seed)
    x = randn(g, rows, cols, std=std, mean=mean, dtype=dtype) if x is None else x
    w = randn(g, cols, std=0.2, mean=1.0, dtype=dtype) if weight else None
    b = randn(g, cols, std=0.2, dtype=dtype) if bias else None
    dy, dres = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype) if residual else None
    y = x.clone() if "y" in in_place else torch.full_like(x, 7.0)
    mu, rs = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    L.liger_layernorm_fwd(y if "y" in in_place else x, w, b, y, mean=mu, rstd=rs, eps=eps)
    ry, mag, rm, rr = fwd_ref(x, w, b, eps)
    c = _chain(cols)
    check(y, ry, mag, c, "y")
    check(mu, rm, x.double().abs().mean(1) if cols else rm, c, "mean")
    check(rs, rr, rr, c, "rstd")
    dx = dy.clone() if "dy" in in_place else dres.clone() if "dres" in in_place else torch.full_like(x, 7.0)
    dw = torch.full((cols,), 7.0, dtype=dtype, device="cuda") if weight else None
    db = torch.full((cols,), 7.0, dtype=dtype, device="cuda") if bias else None
    ws = torch.full((L.liger_layernorm_bwd_workspace(rows, cols) + 64,), 255, dtype=torch.uint8, device="cuda")
    L.liger_layernorm_bwd(dx if "dy" in in_place else dy, x, w, mu, rs, dx, dw, db, ws[:-64],
                          dres=dx if "dres" in in_place else dres)
    assert bool((ws[-64:] == 255).all())
    rdx, mdx, rdw, mdw, rdb, mdb = bwd_ref(dy, dres, x, w, mu, rs)
    check(dx, rdx, mdx, c, "dx")
    tree = rows / 64 + 150      # a block's run of rows, then its partial rows
    if weight:
        check(dw, rdw, mdw, tree, "dw")
    if bias:
        check(db, rdb, mdb, tree, "db")
    return y, dx, dw, db


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (1, 8), (2, 7), (5, 33), (7, 64), (4, 255), (9, 256), (33, 1000), (300, 1001),
                                       (2, 4096), (1111, 768), (640, 4096), (50, 5120), (20, 8200), (9, 16384), (5, 20011), (3, 40000),
                                       (2, 70000), (1, 131072)])
def test_shapes(cuda_lib, dtype, rows, cols):
    run_case(cuda_lib, dtype, rows, cols, seed=rows * 7 + cols)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("parts", [(False, False, False), (True, False, True), (False, True, False), (True, True, False)])
@pytest.mark.parametrize("rows,cols", [(70, 512), (13, 77), (5, 12000)])
def test_optional_parts(cuda_lib, dtype, parts, rows, cols):
    w, b, r = parts
    run_case(cuda_lib, dtype, rows, cols, weight=w, bias=b, residual=r)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(40, 1024), (11, 131), (3, 30000)])
@pytest.mark.parametrize("alias", ["y dy", "y dres"])
def test_in_place_gives_the_same_bits(cuda_lib, dtype, rows, cols, alias):
    a = run_case(cuda_lib, dtype, rows, cols, seed=5)
    b = run_case(cuda_lib, dtype, rows, cols, seed=5, in_place=alias)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(9001, 131), (7003, 333), (5001, 515), (3001, 1001), (2003, 1999), (2001, 2050), (1501, 4097), (901, 4099),
                                       (903, 6001), (801, 8185), (801, 8191), (701, 12345), (607, 16001)])
def test_many_rows_of_odd_width(cuda_lib, dtype, rows, cols):
    """More rows than blocks: a block goes on to rows that start at the same place of their 16-byte windows."""
    run_case(cuda_lib, dtype, rows, cols, seed=rows + cols)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(3001, 1001), (1501, 4097)])
@pytest.mark.parametrize("alias", ["y dy", "y dres"])
def test_many_rows_of_odd_width_in_place(cuda_lib, dtype, rows, cols, alias):
    a = run_case(cuda_lib, dtype, rows, cols, seed=6)
    b = run_case(cuda_lib, dtype, rows, cols, seed=6, in_place=alias)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [512, 777, 9000])
def test_rows_far_from_zero_and_of_any_size(cuda_lib, dtype, cols):
    # a mean 300 times the spread: E x^2 - mean^2 would lose all of the variance's digits
    run_case(cuda_lib, dtype, 17, cols, std=1.0, mean=300.0)
    run_case(cuda_lib, dtype, 17, cols, std=1e-6, mean=0.0, eps=0.0)
    run_case(cuda_lib, dtype, 17, cols, std=1e6, mean=-1e6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [256, 77, 20000])
def test_constant_rows_give_the_bias(cuda_lib, dtype, cols):
    import transformer_rmsnorm_fwd_gb300 as L
    x = torch.full((3, cols), 3.0, dtype=dtype, device="cuda")
    w, b = torch.full_like(x[0], 2.0), torch.linspace(-1, 1, cols, device="cuda").to(dtype)
    y, mu, rs = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    L.liger_layernorm_fwd(x, w, b, y, mean=mu, rstd=rs, eps=1e-5)
    assert torch.equal(mu, torch.full_like(mu, 3.0))        # (the sum of up to 20000 threes is exact in fp32)
    assert torch.equal(y, b.expand_as(y))
    check(rs, torch.full((3,), 1e-5 ** -0.5, dtype=torch.float64, device="cuda"), rs.double(), 4, "rstd")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [320, 101, 9000])
def test_infinities_and_nan_stay_in_their_rows(cuda_lib, dtype, cols):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(3)
    x = randn(g, 6, cols, dtype=dtype)
    clean = x.clone()
    x[1, cols // 2], x[3, 0], x[4, cols - 1] = float("nan"), float("inf"), float("-inf")
    y, z = torch.empty_like(x), torch.empty_like(x)
    L.liger_layernorm_fwd(x, None, None, y)
    L.liger_layernorm_fwd(clean, None, None, z)
    for r in (0, 2, 5):
        assert torch.equal(y[r], z[r])
    for r in (1, 3, 4):
        assert bool(torch.isnan(y[r]).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows(cuda_lib, dtype):
    import transformer_rmsnorm_fwd_gb300 as L
    x = torch.empty(0, 40, dtype=dtype, device="cuda")
    mu = torch.empty(0, device="cuda")
    dw, db = (torch.full((40,), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    L.liger_layernorm_fwd(x, dw, db, x, mean=mu, rstd=mu)
    L.liger_layernorm_bwd(x, x, dw, mu, mu, x, dw, db, None)
    assert not dw.any() and not db.any()


def test_gradient_against_differences(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(11)
    rows, cols, eps = 4, 24, 1e-2
    x, w, b, dy = (randn(g, *s) for s in ((rows, cols), (cols,), (cols,), (rows, cols)))
    mu, rs, y = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(L.liger_layernorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    L.liger_layernorm_fwd(x, w, b, y, mean=mu, rstd=rs, eps=eps)
    L.liger_layernorm_bwd(dy, x, w, mu, rs, dx, dw, db, ws)

    def loss(x, w, b):
        return float((fwd_ref(x, w, b, eps)[0] * dy.double()).sum())

    h = 1e-5        # central differences of the formula in 64 bits: h^2 of the third derivative, and 1e-16 / h
    for t, d, other in ((x, dx, lambda v: (v, w, b)), (w, dw, lambda v: (x, v, b)), (b, db, lambda v: (x, w, v))):
        for i in range(0, t.numel(), 7):
            up, down = t.double().clone(), t.double().clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            diff = (loss(*other(up)) - loss(*other(down))) / (2 * h)
            assert abs(diff - float(d.view(-1)[i])) < 2e-5 * (1 + abs(diff)), i


def test_refusals(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    x = torch.zeros(4, 64, device="cuda")
    y, r = torch.empty_like(x), torch.empty(4, device="cuda")
    for bad in (dict(w=torch.zeros(63, device="cuda")), dict(w=torch.zeros(64, device="cuda", dtype=torch.bfloat16)),
                dict(x=x.t()), dict(y=torch.empty(4, 63, device="cuda")), dict(x=x.cpu()), dict(mean=torch.empty(3, device="cuda")),
                dict(x=x.half(), y=y.half(), w=None)):
        a = dict(dict(x=x, w=x[0], b=None, y=y, mean=r, rstd=None), **bad)
        with pytest.raises((ValueError, TypeError)):
            L.liger_layernorm_fwd(a["x"], a["w"], a["b"], a["y"], mean=a["mean"], rstd=a["rstd"])
    with pytest.raises(L.LigerError):
        L.liger_layernorm_fwd(x, None, None, y, eps=-1.0)
    with pytest.raises(L.LigerError):
        L.liger_layernorm_bwd(x, x, None, r, r, y, x[0].clone(), None, torch.empty(16, dtype=torch.uint8, device="cuda"))
