"""Helpers of the post-training operators' tests: the error bound an output is held to.

A floating output may be off its 64-bit value by half a step of its storage type, u |ref| (u = finfo.eps / 2), and by the
fp32 arithmetic before it: a chain of n roundings of 2^-24 each on terms whose magnitudes add up to `mag`."""
import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, mag, chain, what):
    """|got - ref| <= u |ref| + chain 2^-24 mag (1 + u), element by element; NaN and infinities in the same places."""
    u = half_step(got.dtype)
    g, ref, mag = got.double(), ref.double(), mag.double()
    assert g.shape == ref.shape, what
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(g), fine), what
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), what
    bound = u * ref.abs() + chain * U32 * mag * (1 + u) + 2.0 ** -126
    over = ((g - ref).abs() - bound)[fine]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: off by {worst:.3e} more than allowed ({int((over > 0).sum())} of {over.numel()})"
