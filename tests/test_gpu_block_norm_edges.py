"""Block norms at the ends of the range: infinities in z where the formulas do not let them reach a gradient, on every kernel
(staged rows, odd widths, the generic kernel), against the definition in 64 bits."""
import pytest
import torch

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
