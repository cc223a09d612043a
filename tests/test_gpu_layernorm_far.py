"""Layer norm of fp32 rows whose mean is many deviations from 0: the output's error is that of the differences, not of the mean."""
import pytest
import torch

from layer_util import gen, randn
from train_util import U32, check

pytestmark = pytest.mark.gpu


# rows held by teams of warps, one element or a vector a time; rings of whole vectors, several teams a block and one; rows of odd
# width, few and many; rows too wide for any of these
@pytest.mark.parametrize("rows,cols", [(4, 4096), (9, 77), (30, 8192), (2000, 128), (5000, 512), (700, 4096), (330, 8000), (300, 131),
                                       (6000, 333), (3001, 1001), (901, 4099), (310, 6001), (40, 8185), (5, 20011), (3, 40000)])
@pytest.mark.parametrize("mean,std", [(1000.0, 1.0), (-1e5, 1.0), (3e-3, 1e-6)])
def test_a_large_mean_costs_no_digits(cuda_lib, rows, cols, mean, std):
    """x - m is exact for x near m, whatever m was rounded to, and so only the sums of these differences round: cols / 32 terms in a
    register, a tree, and a few roundings of the result.  They are of the size of x - mean and of mean - m, which is the same number of
    roundings of mean |x|, one order further down."""
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(rows + cols)
    x = randn(g, rows, cols, std=std, mean=mean)
    w, b = randn(g, cols, std=0.2, mean=1.0), randn(g, cols, std=0.2)
    y, mu, rs = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    eps = 1e-14
    L.liger_layernorm_fwd(x, w, b, y, mean=mu, rstd=rs, eps=eps)
    x = x.double()
    m = x.mean(1, keepdim=True)
    d = x - m
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    chain = cols / 32 + 40
    off = chain * U32 * x.abs().mean(1, keepdim=True)
    size = d.abs() + d.abs().mean(1, keepdim=True) + off
    check(y, d * rstd * w.double() + b.double(), size * rstd * w.double().abs() + b.double().abs(), chain, "y")
    check(mu, m[:, 0], d.abs().mean(1) + off[:, 0], chain, "mean")
    check(rs, rstd[:, 0], rstd[:, 0], chain, "rstd")
