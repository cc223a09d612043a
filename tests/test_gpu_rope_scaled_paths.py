"""The scaled rotation gives the same bits whichever way its elements travel: staged, in whole chunks, or one by one."""
import pytest
import torch

from layer_util import gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("B,S,Hq,Hk,D,R", [(2, 20, 2, 1, 2, 2), (3, 400, 8, 1, 4, 2), (2, 300, 4, 2, 64, 32), (1, 1000, 5, 3, 80, 20), (1, 9, 32, 8, 128, 128)])
def test_alignment_does_not_change_bits(cuda_lib, dtype, pairing, B, S, Hq, Hk, D, R):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(S + D)
    packed = randn(g, B, S, Hq + Hk, D, dtype=dtype)
    args = dict(pairing=pairing, scaling="ntk", factor=8.0)

    def run(offset, in_place):
        """The same q and k with the outputs `offset` elements into their buffers."""
        x = torch.empty(packed.numel() + 16, dtype=dtype, device="cuda")[offset:offset + packed.numel()].view(packed.shape)
        x.copy_(packed)
        q, k = x[:, :, :Hq], x[:, :, Hq:]
        if in_place:
            L.liger_rope_scaled_fwd(q, k, q, k, R, **args)
            return q, k
        outs = [torch.empty(B * S * h * D + 16, dtype=dtype, device="cuda")[offset:offset + B * S * h * D].view(B, S, h, D) for h in (Hq, Hk)]
        L.liger_rope_scaled_fwd(q, k, *outs, R, **args)
        return outs

    ways = [run(o, p) for o in (0, 1, 8) for p in (False, True)]
    for q, k in ways[1:]:
        assert torch.equal(q, ways[0][0]) and torch.equal(k, ways[0][1])
