"""Block norms at the ends of the range: infinities in z where the formulas do not let them reach a gradient, and rows far from 1
in size, on every kernel (staged rows, odd widths, the generic kernel), against the definition in 64 bits."""
import pytest
import torch

import test_gpu_block_norm
from test_gpu_block_norm import L, _backward, _bwd64, _make   # noqa: F401
from train_util import check

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
# staged with one team and with several, odd widths in one and in more blocks, generic (narrow odd, wide)
@pytest.mark.parametrize("rows,cols,gates", [(40, 4096, 1), (40, 4096, 40), (300, 256, 3), (30, 8192, 2), (40, 1001, 1),
                                             (40, 1001, 40), (12, 4095, 2), (12, 37, 1), (6, 20000, 2)])
@pytest.mark.parametrize("pre", [True, False])
def test_dz_without_post_norm_does_not_depend_on_z(L, rows, cols, gates, dtype, pre):  # noqa: F811
    """dz = block_scale g D without w_post: an infinity or NaN in z reaches the gate's gradient in its column and nothing else."""
    d = _make(rows, cols, dtype, False, gates, pre, seed=11)
    h = d["r"]
    rh = (h.double().square().mean(1) + EPS).rsqrt().float() if pre else None
    ref, mag = _bwd64(d, h, 0.9, 0.7, rows, gates)
    bad = {1: float("inf"), cols // 2: float("-inf"), cols - 1: float("nan")}
    for k, (c, v) in enumerate(bad.items()):
        d["z"][(k * 2 + 1) % rows, c] = v
    got = _backward(L, d, h, None, rh, 0.9, 0.7, rows, gates)
    chain = cols / 32 + 60
    for k in ("dr", "dz"):
        check(got[k], ref[k], mag[k], chain, k)
    if pre:
        check(got["dw_pre"], ref["dw_pre"], mag["dw_pre"], chain + rows + 64, "dw_pre")
    clean = torch.ones(cols, dtype=torch.bool, device="cuda")
    clean[list(bad)] = False
    check(got["dgate"][:, clean], ref["dgate"][:, clean], mag["dgate"][:, clean], chain + rows + 64, "dgate")
    rows_of = rows // gates
    for k, c in enumerate(bad):
        at = (k * 2 + 1) % rows // rows_of
        col = torch.isfinite(got["dgate"][:, c].double())
        assert not bool(col[at]) and int(col.sum()) == gates - 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(40, 4096), (300, 256), (40, 1001), (12, 37), (6, 20000)])
@pytest.mark.parametrize("h_size,z_size", [(1e15, 1.0), (1e17, 1.0), (1e-15, 1.0), (1.0, 1e15), (1.0, 1e17), (1.0, 1e-15)])
def test_rows_far_from_one(L, monkeypatch, rows, cols, dtype, h_size, z_size):  # noqa: F811
    """The scale of a row of size s is 1 / s, and its third power leaves fp32's range long before the gradients do."""
    monkeypatch.setattr(test_gpu_block_norm, "EPS", 0.0)
    d = _make(rows, cols, dtype, True, 1, True, seed=12)
    d["dh"] = None
    d["z"] = (d["z"].double() * z_size).to(d["z"].dtype)
    h = (d["r"].double() * h_size).to(d["r"].dtype)
    rz, rh = (x.double().square().mean(1).rsqrt().float() for x in (d["z"], h))
    ref, mag = _bwd64(d, h, 1.0, 0.7, rows, 1)
    got = _backward(L, d, h, rz, rh, 1.0, 0.7, rows, 1)
    for k, v in got.items():
        chain = cols / 32 + 60
        check(v, ref[k], mag[k], chain if k in ("dr", "dz") else chain + rows + 64, k)
