"""What liger_device_status says of an expired wait of the layer-norm layer's operators, which share the words of others."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which,names", [(0, ("RMSNorm", "block norm", "layer norm")), (1, ("FusedLinearSwiGLU", "projections")),
                                         (3, ("RoPE", "scaled RoPE"))])
def test_a_shared_word_names_all_that_share_it(cuda_lib, which, names):
    cuda_lib.liger_device_status()
    cuda_lib.liger_device_status_mark(which)
    with pytest.raises(cuda_lib.LigerError) as e:
        cuda_lib.liger_device_status()
    assert all(n in str(e.value) for n in names)


def test_all_words_fit_the_message(cuda_lib):
    for which in range(4):
        cuda_lib.liger_device_status_mark(which)
    with pytest.raises(cuda_lib.LigerError) as e:
        cuda_lib.liger_device_status()
    assert all(n in str(e.value) for n in ("layer norm", "projections", "QKV", "scaled RoPE", "incomplete"))
    cuda_lib.liger_device_status()


def test_words_are_clear_after_normal_calls(cuda_lib):
    import torch
    import transformer_rmsnorm_fwd_gb300 as L
    x, w = torch.randn(700, 4096, device="cuda").bfloat16(), torch.randn(512, 4096, device="cuda").bfloat16()
    y, out = torch.empty_like(x), torch.empty(700, 512, dtype=torch.bfloat16, device="cuda")
    L.liger_layernorm_fwd(x, None, None, y)
    L.liger_linear_act_fwd(x, w, out)
    L.liger_linear_act_fwd(x[:4].contiguous(), w, out[:4])
    q = x.view(1, 700, 32, 128)
    L.liger_rope_scaled_fwd(q, None, torch.empty_like(q), None, 64)
    cuda_lib.liger_device_status()
