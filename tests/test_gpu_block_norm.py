"""liger_block_norm_fwd / _bwd against the definition in 64 bits (the backward by automatic differentiation of the forward,
and against differences of it): widths with and without whole 16-byte vectors, one row to some thousand, every combination
of post-norm, gate and pre-norm, gate rows shared by one row to all, in place, rows of zeros and infinities.

The longest chain of fp32 roundings: a row's sum takes at most cols / 32 adds in one thread and some 40 more across threads
and in the formulas; a sum over rows at most one add for each row and 64 more."""
import pytest
import torch

from train_util import check

pytestmark = pytest.mark.gpu
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def L(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as lib
    return lib


def _make(rows, cols, dtype, post, gates, pre, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]

    def rnd(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, device="cuda", generator=g) * std + mean).to(dt)
    return {"z": rnd(rows, cols), "r": rnd(rows, cols, std=1.5), "dh": rnd(rows, cols), "dy": rnd(rows, cols) if pre else None,
            "w_post": rnd(cols, std=0.2, mean=1.0) if post else None, "w_pre": rnd(cols, std=0.2, mean=1.0) if pre else None,
            "gate": rnd(gates, cols, std=0.5, mean=0.3) if gates else None}


def _fwd64(d, a, b, rows, gates):
    f = {k: v.double() if v is not None else None for k, v in d.items()}
    p, rz, rh, y = f["z"], None, None, None
    if f["w_post"] is not None:
        rz = (p.square().mean(1) + EPS).rsqrt()
        p = p * rz[:, None] * f["w_post"]
    if gates:
        p = p * f["gate"].repeat_interleave(rows // gates, 0)
    h = a * f["r"] + b * p
    if f["w_pre"] is not None:
        rh = (h.square().mean(1) + EPS).rsqrt()
        y = h * rh[:, None] * f["w_pre"]
    return h, y, rz, rh, a * f["r"].abs() + abs(b) * p.abs()


def _forward(L, d, a, b, rows, in_place=False):
    z = d["z"].clone() if in_place else d["z"]
    r = d["r"].clone() if in_place else d["r"]
    h = r if in_place else torch.full_like(z, 7.0)
    y = None if d["w_pre"] is None else z if in_place else torch.full_like(z, 7.0)
    rz, rh = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    L.liger_block_norm_fwd(z, r, h, y, d["w_post"], d["gate"], d["w_pre"], rz, rh, a, b, EPS)
    return h, y, rz, rh


SHAPES = [(1, 1), (1, 4096), (3, 64), (5, 33), (257, 1001), (64, 8192), (7, 520), (300, 4096), (2, 16384), (4, 20000),
          (1000, 256), (33, 2050), (1, 65), (700, 129), (400, 1023), (301, 3001), (330, 4095), (200, 5003), (160, 8191), (400, 2047),
          # rows enough for every form of the staged kernels: several teams a block, one, wide rows
          (5000, 256), (3000, 512), (2500, 640), (320, 1536), (330, 5120), (400, 8192), (170, 12288), (170, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(L, rows, cols, dtype):
    for post, gates, pre, a, b in [(True, 1, True, 1.0, 1.0), (True, 0, True, 0.7, 1.3), (False, 1, True, 1.0, -0.5),
                                   (True, rows, True, 1.0, 1.0), (True, 1, False, 1.0, 0.25), (False, 0, False, 0.5, 2.0),
                                   (False, 0, True, 1.0, 1.0)]:
        d = _make(rows, cols, dtype, post, gates, pre)
        for in_place in (False, True):
            h, y, rz, rh = _forward(L, d, a, b, rows, in_place)
            h64, y64, rz64, rh64, mag = _fwd64(d, a, b, rows, gates)
            chain = cols / 32 + 40
            check(h, h64, mag, chain, "h")
            if post:
                check(rz, rz64, rz64.abs(), chain, "rstd_z")
            else:
                assert bool((rz == 7.0).all())
            if pre:
                # h's own error (chain roundings of mag) passes to rh through the row's norm and to y
                scale = (mag.square().mean(1) + EPS).sqrt() * rh64
                check(rh, rh64, rh64 * scale, 2 * chain, "rstd_h")
                w = d["w_pre"].double().abs()
                check(y, y64, (mag * rh64[:, None] + h64.abs() * (rh64 * scale)[:, None]) * w, 2 * chain, "y")
            else:
                assert bool((rh == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,gates", [(3000, 1024, 6), (3000, 1024, 750), (6000, 256, 1500), (6000, 512, 2000),
                                             (400, 4096, 8), (400, 4096, 200), (336, 6144, 7), (1200, 1001, 300), (900, 77, 90)])
def test_forward_gate_rows(L, rows, cols, gates, dtype):
    """Gate rows shared by some rows, that teams of warps meet in every order."""
    d = _make(rows, cols, dtype, True, gates, True, seed=4)
    h, y, rz, rh = _forward(L, d, 1.0, 0.8, rows)
    h64, y64, rz64, rh64, mag = _fwd64(d, 1.0, 0.8, rows, gates)
    chain = cols / 32 + 40
    check(h, h64, mag, chain, "h")
    scale = (mag.square().mean(1) + EPS).sqrt() * rh64
    check(y, y64, (mag * rh64[:, None] + h64.abs() * (rh64 * scale)[:, None]) * d["w_pre"].double().abs(), 2 * chain, "y")


def _bwd64(d, h, a, b, rows, gates):
    """Gradients by automatic differentiation in 64 bits, and the magnitudes that their sums are made of."""
    f = {k: v.double() if v is not None else None for k, v in d.items()}
    H = h.shape[1]
    h = h.double().requires_grad_()
    leaf = {k: f[k].clone().requires_grad_() for k in ("z", "w_post", "gate", "w_pre") if f[k] is not None}
    top = (f["dh"] * h).sum() if f["dh"] is not None else 0.0
    rh = rz = None
    if f["w_pre"] is not None:
        rh = (h.square().mean(1) + EPS).rsqrt()
        top = top + (f["dy"] * h * rh[:, None] * leaf["w_pre"]).sum()
    D, = torch.autograd.grad(top, h, retain_graph=True)
    out = {"dr": a * D}
    if rh is not None:
        out["dw_pre"], = torch.autograd.grad(top, leaf["w_pre"])
    p = leaf["z"]
    if f["w_post"] is not None:
        rz = (p.square().mean(1) + EPS).rsqrt()
        p = p * rz[:, None] * leaf["w_post"]
    if gates:
        p = p * leaf["gate"].repeat_interleave(rows // gates, 0)
    names = [k for k in ("z", "w_post", "gate") if k in leaf]
    for k, g in zip(names, torch.autograd.grad((b * D * p).sum(), [leaf[k] for k in names])):
        out["d" + k] = g
    with torch.no_grad():
        mag = {}
        M = f["dh"].abs() if f["dh"] is not None else torch.zeros_like(h)
        if rh is not None:
            u = (f["dy"] * f["w_pre"]).abs()
            M = M + rh[:, None] * u + h.abs() * (rh ** 3 / H * (u * h.abs()).sum(1))[:, None]
            mag["dw_pre"] = (f["dy"] * h * rh[:, None]).abs().sum(0)
        mag["dr"] = abs(a) * M
        z = f["z"].abs()
        q = torch.full_like(M, abs(b))
        if gates:
            q = q * f["gate"].abs().repeat_interleave(rows // gates, 0)
        s = M * z * (rz[:, None] if rz is not None else 1.0)
        if gates:
            w = f["w_post"].abs() if f["w_post"] is not None else 1.0
            mag["dgate"] = (abs(b) * s * w).view(gates, -1, H).sum(1)
        if rz is not None:
            mag["dw_post"] = (q * s).sum(0)
            q = q * f["w_post"].abs()
            mag["dz"] = q * M * rz[:, None] + z * (rz ** 3 / H * (q * M * z).sum(1))[:, None]
        else:
            mag["dz"] = q * M
    return out, mag


def _backward(L, d, h, rz, rh, a, b, rows, gates, in_place=False):
    cols = h.shape[1]
    dh = d["dh"].clone() if in_place and d["dh"] is not None else d["dh"]
    dy = d["dy"].clone() if in_place and d["dy"] is not None else d["dy"]
    dr = dh if in_place and dh is not None else torch.full_like(h, 7.0)
    dz = dy if in_place and dy is not None else torch.full_like(h, 7.0)
    ws = torch.full((max(L.liger_block_norm_bwd_workspace(rows, cols, gates), 16),), 255, dtype=torch.uint8, device="cuda")
    g = {"d" + k: torch.full_like(d[k], 7.0) if d[k] is not None else None for k in ("w_post", "gate", "w_pre")}
    L.liger_block_norm_bwd(dh, dy, d["z"], h, dr, dz, ws, d["w_post"], d["gate"], d["w_pre"], rz, rh, g["dw_post"],
                           g["dgate"], g["dw_pre"], a, b)
    return {"dr": dr, "dz": dz, **{k: v for k, v in g.items() if v is not None}}


def _bwd_case(L, rows, cols, dtype, post, gates, pre, a, b, grad_h=True, in_place=False, seed=1):
    d = _make(rows, cols, dtype, post, gates, pre, seed)
    if not grad_h:
        d["dh"] = None
    h = d["r"]
    rz = (d["z"].double().square().mean(1) + EPS).rsqrt().float() if post else None
    rh = (h.double().square().mean(1) + EPS).rsqrt().float() if pre else None
    ref, mag = _bwd64(d, h, a, b, rows, gates)
    got = _backward(L, d, h, rz, rh, a, b, rows, gates, in_place)
    assert set(got) == set(ref)
    for k, v in got.items():
        row_chain = cols / 32 + 60
        check(v, ref[k], mag[k], row_chain if k in ("dr", "dz") else row_chain + rows + 64, f"{k} {rows}x{cols}")
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(L, rows, cols, dtype):
    for n, (post, gates, pre, a, b, grad_h) in enumerate([
            (True, 1, True, 1.0, 1.0, True), (True, 0, True, 0.7, 1.3, True), (False, 1, True, 1.0, -0.5, False),
            (True, rows, True, 1.0, 1.0, True), (True, 1, False, 1.0, 0.25, True), (False, 0, False, 0.5, 2.0, True),
            (False, 0, True, 1.0, 1.0, True), (True, 0, True, 1.0, 1.0, False)]):
        _bwd_case(L, rows, cols, dtype, post, gates, pre, a, b, grad_h, in_place=n % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,gates", [(12, 3), (1200, 4), (1200, 100), (1500, 750), (2000, 2000), (3000, 1500), (640, 160)])
@pytest.mark.parametrize("cols", [256, 77, 1500])
def test_backward_gate_rows(L, rows, gates, cols, dtype):
    """Gate rows shared by many rows (their sums split over blocks), by two, by one."""
    _bwd_case(L, rows, cols, dtype, True, gates, True, 1.0, 0.5)
    _bwd_case(L, rows, cols, dtype, False, gates, True, 1.0, 0.5)


@pytest.mark.parametrize("rows,cols", [(1, 64), (40, 96), (6, 37)])
def test_backward_against_differences(L, rows, cols):
    """<gradient, v> is the slope of the 64-bit forward along v."""
    d = _make(rows, cols, "f32", True, 2 if rows % 2 == 0 else 1, True, seed=3)
    gates, a, b = d["gate"].shape[0], 0.8, 1.2
    h, y, rz, rh = _forward(L, d, a, b, rows)
    d64 = {k: v.double() for k, v in d.items()}
    got = _backward(L, d, h, rz, rh, a, b, rows, gates)

    def value(x):
        h64, y64, *_ = _fwd64(x, a, b, rows, gates)
        return float((h64 * d64["dh"]).sum() + (y64 * d64["dy"]).sum())
    gen = torch.Generator(device="cuda").manual_seed(9)
    for name, grad in (("z", "dz"), ("r", "dr"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_pre", "dw_pre")):
        v = torch.randn(d64[name].shape, device="cuda", generator=gen, dtype=torch.float64)
        up, down = dict(d64), dict(d64)
        up[name], down[name] = d64[name] + 1e-6 * v, d64[name] - 1e-6 * v
        slope = (value(up) - value(down)) / 2e-6
        # the differences are good to about 1e-9 of the values' size; h was rounded to fp32 (2^-24)
        size = float((got[grad].double().abs() * v.abs()).sum())
        assert abs(float((got[grad].double() * v).sum()) - slope) <= 1e-5 * size + 1e-7 * abs(value(d64)), name


def test_runs_are_the_same_bits(L):
    d = _make(700, 1024, "bf16", True, 7, True)
    rz = (d["z"].double().square().mean(1) + EPS).rsqrt().float()
    rh = (d["r"].double().square().mean(1) + EPS).rsqrt().float()
    one = _backward(L, d, d["r"], rz, rh, 1.0, 1.0, 700, 7)
    two = _backward(L, d, d["r"], rz, rh, 1.0, 1.0, 700, 7)
    for k in one:
        assert torch.equal(one[k], two[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [4096, 513])
def test_zero_and_infinite_rows(L, dtype, cols):
    """A row of zeros is scaled by 1/sqrt(eps); infinities and NaN stay in their own rows."""
    d = _make(9, cols, dtype, True, 1, True)
    d["z"][2], d["r"][2] = 0, 0
    d["z"][4, 1], d["r"][6, 3] = float("inf"), float("nan")
    h, y, rz, rh = _forward(L, d, 1.0, 1.0, 9)
    h64, y64, rz64, rh64, mag = _fwd64(d, 1.0, 1.0, 9, 1)
    good = torch.tensor([0, 1, 2, 3, 5, 7, 8], device="cuda")
    check(h[good], h64[good], mag[good], cols / 32 + 40, "h")
    assert bool((y[2] == 0).all()) and abs(float(rh[2]) * EPS ** 0.5 - 1) < 1e-6
    assert bool(torch.isfinite(y[good].double()).all())
    assert bool(torch.isnan(y[4]).any()) and bool(torch.isnan(y[6]).all())
    got = _backward(L, d, h, rz, rh, 1.0, 1.0, 9, 1)
    assert bool(torch.isfinite(got["dz"][good].double()).all())


def test_no_rows(L):
    d = _make(0, 256, "bf16", True, 0, True)
    h, y, _, _ = _forward(L, d, 1.0, 1.0, 0)
    assert h.shape == (0, 256)
    got = _backward(L, d, d["r"], torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), 1.0, 1.0, 0, 0)
    assert bool((got["dw_post"] == 0).all()) and bool((got["dw_pre"] == 0).all())


def test_refusals(L):
    d = _make(6, 64, "bf16", True, 1, True)
    h, y = torch.empty_like(d["z"]), torch.empty_like(d["z"])
    ok = dict(w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    with pytest.raises(ValueError):
        L.liger_block_norm_fwd(d["z"].t().contiguous().t(), d["r"], h, y, **ok)      # not contiguous
    with pytest.raises(ValueError):
        L.liger_block_norm_fwd(d["z"], d["r"][:5], h, y, **ok)
    with pytest.raises(ValueError):
        L.liger_block_norm_fwd(d["z"].cpu(), d["r"], h, y, **ok)
    with pytest.raises(TypeError):
        L.liger_block_norm_fwd(d["z"], d["r"].float(), h, y, **ok)
    with pytest.raises(ValueError):
        L.liger_block_norm_fwd(d["z"], d["r"], h, y, **{**ok, "w_post": d["w_post"][:32].clone()})
    with pytest.raises(L.LigerError) as e:      # 4 gate rows for 6 rows
        L.liger_block_norm_fwd(d["z"], d["r"], h, y, **{**ok, "gate": d["gate"].expand(4, 64).contiguous()})
    assert e.value.status == -2
    with pytest.raises(L.LigerError) as e:      # y missing
        L.liger_block_norm_fwd(d["z"], d["r"], h, None, **ok)
    assert e.value.status == -1
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(L.LigerError) as e:
        L.liger_block_norm_bwd(d["dh"], d["dy"], d["z"], h, torch.empty_like(h), torch.empty_like(h), ws, **ok,
                               rstd_z=torch.empty(6, device="cuda"), rstd_h=torch.empty(6, device="cuda"),
                               dw_post=d["w_post"], dgate=d["gate"], dw_pre=d["w_pre"])
    assert e.value.status == -6
