"""Partial rotary positions with scaled frequencies against their formulas in 64 bits: pairings, head sizes, strides, in place."""
import pytest
import torch

from layer_util import frequencies, gen, randn, rotate
from train_util import check

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
SCALINGS = {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=8.0), "bands": dict(factor=8.0, low=1.0, high=4.0, orig_len=512.0),
            "yarn": dict(factor=16.0, low=1.0, high=32.0, orig_len=1024.0)}
CHAIN = 16      # the angle rounded to fp32 (up to pi 2^-24), cos and sin (2 ulp), their product with m, two products and a sum


def _tensors(g, dtype, B, S, Hq, Hk, D, packed):
    if packed:      # q, k and v of a token stand side by side
        buf = randn(g, B, S, Hq + 2 * Hk, D, dtype=dtype)
        return buf[:, :, :Hq], buf[:, :, Hq:Hq + Hk]
    return randn(g, B, S, Hq, D, dtype=dtype), randn(g, B, S, Hk, D, dtype=dtype)


def _positions(g, B, S, far):
    return None if far is None else torch.randint(-far, far, (B, S), device="cuda", generator=g).to(torch.int32)


def run_case(dtype, B, S, Hq, Hk, D, R, pairing="half", scaling="none", theta=1e4, far=None, packed=False, attn_factor=0.0, seed=0):
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(seed)
    q, k = _tensors(g, dtype, B, S, Hq, Hk, D, packed)
    pos = _positions(g, B, S, far)
    p = torch.arange(S, device="cuda").expand(B, S) if pos is None else pos
    args = dict(pos=pos, theta=theta, pairing=pairing, scaling=scaling, attn_factor=attn_factor, **SCALINGS[scaling])
    f, m = frequencies(R, theta, scaling, attn_factor=attn_factor, **SCALINGS[scaling])
    outs = []
    for fn, sign in ((L.liger_rope_scaled_fwd, 1.0), (L.liger_rope_scaled_bwd, -1.0)):
        qo, ko = (torch.full((B, S, h, D), 7.0, dtype=dtype, device="cuda") for h in (Hq, Hk))
        fn(q, k, qo, ko, R, **args)
        for x, o in ((q, qo), (k, ko)):
            ref, mag = rotate(x.double(), p, f, m, R, pairing, sign)
            check(o, ref, mag, CHAIN, "rotated")
            assert torch.equal(o[..., R:], x[..., R:])
        outs += [qo, ko]
        # in place on the same views: the same bits, and nothing else of the buffer changed
        buf_q, buf_k = _tensors(gen(seed), dtype, B, S, Hq, Hk, D, packed)
        v0 = buf_q._base[:, :, Hq + Hk:].clone() if packed else None
        fn(buf_q, buf_k, buf_q, buf_k, R, **args)
        assert torch.equal(buf_q, qo) and torch.equal(buf_k, ko)
        if packed:
            assert torch.equal(buf_q._base[:, :, Hq + Hk:], v0)
    return outs


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (64, 16), (80, 32), (80, 20), (96, 96), (96, 24), (128, 64), (128, 2), (256, 64),
                                 (40, 10), (33, 6), (17, 16), (512, 512), (2, 2), (256, 256)])
def test_head_sizes(cuda_lib, dtype, pairing, D, R):
    run_case(dtype, 2, 5, 6, 2, D, R, pairing, seed=D + R)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("packed", [False, True])
def test_scalings(cuda_lib, dtype, scaling, packed):
    run_case(dtype, 2, 300, 4, 1, 64, 32, "half", scaling, packed=packed)
    run_case(dtype, 3, 1, 4, 4, 128, 128, "interleaved", scaling, theta=5e5, far=1 << 20, packed=packed)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,S,Hq,Hk", [(1, 1, 1, 1), (64, 1, 32, 8), (1, 4099, 3, 1), (7, 13, 1, 5), (3, 130, 40, 8), (2, 9, 70, 70)])
def test_batches(cuda_lib, dtype, B, S, Hq, Hk):
    run_case(dtype, B, S, Hq, Hk, 64, 32, far=(1 << 31) - 1 if S == 1 else None, packed=True, attn_factor=1.25)


@pytest.mark.parametrize("scaling", list(SCALINGS))
def test_two_rotated_elements_and_whole_turns(cuda_lib, scaling):
    run_case(torch.float32, 2, 3, 2, 1, 8, 2, "half", scaling)


def test_transpose(cuda_lib):
    """<fwd(x), g> = <x, bwd(g)>, and bwd undoes fwd up to m^2."""
    import transformer_rmsnorm_fwd_gb300 as L
    g = gen(9)
    x, d = randn(g, 2, 40, 3, 48), randn(g, 2, 40, 3, 48)
    y, dx, back = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    args = dict(theta=1e4, scaling="yarn", **SCALINGS["yarn"])
    L.liger_rope_scaled_fwd(x, None, y, None, 24, **args)
    L.liger_rope_scaled_bwd(d, None, dx, None, 24, **args)
    L.liger_rope_scaled_bwd(y, None, back, None, 24, **args)
    lhs, rhs = (y.double() * d.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(float(lhs - rhs)) <= 2 * CHAIN * 2.0 ** -24 * float((x.abs().double() * d.abs().double()).sum()) * 4
    m = frequencies(24, 1e4, "yarn", **SCALINGS["yarn"])[1]
    ref = x.double().clone()
    ref[..., :24] *= m * m
    mag = ref.abs() + ref.abs().amax(-1, keepdim=True) * 3
    check(back, ref, mag, 2 * CHAIN, "back")


def test_only_q_or_only_k(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    q, k = randn(gen(1), 2, 6, 4, 32), randn(gen(2), 2, 6, 2, 32)
    both = torch.empty_like(q), torch.empty_like(k)
    L.liger_rope_scaled_fwd(q, k, *both, 16)
    a, b = torch.empty_like(q), torch.empty_like(k)
    L.liger_rope_scaled_fwd(q, None, a, None, 16)
    L.liger_rope_scaled_fwd(None, k, None, b, 16)
    assert torch.equal(a, both[0]) and torch.equal(b, both[1])
    L.liger_rope_scaled_fwd(q, k, q, b.zero_(), 16)         # one in place, one not
    assert torch.equal(q, both[0]) and torch.equal(b, both[1])


def test_infinities_and_nan_stay_in_their_pairs(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    for dtype in DTYPES:
        x = randn(gen(4), 1, 9, 2, 64, dtype=dtype)
        clean = torch.empty_like(x)
        L.liger_rope_scaled_fwd(x, None, clean, None, 32)
        x[0, 3, 1, 5], x[0, 4, 0, 40], x[0, 5, 0, 20] = float("nan"), float("inf"), float("nan")
        y = torch.empty_like(x)
        L.liger_rope_scaled_fwd(x, None, y, None, 32)
        hit = torch.zeros_like(x, dtype=torch.bool)
        hit[0, 3, 1, [5, 21]] = hit[0, 5, 0, [20, 4]] = hit[0, 4, 0, 40] = True
        assert torch.equal(y[~hit], clean[~hit])
        assert bool(torch.isnan(y[0, 3, 1, [5, 21]]).all()) and float(y[0, 4, 0, 40]) == float("inf")


def test_refusals(cuda_lib):
    import transformer_rmsnorm_fwd_gb300 as L
    q = torch.zeros(2, 3, 4, 16, device="cuda")
    o = torch.empty_like(q)
    for bad in (dict(q=q.transpose(1, 2)), dict(q=q[..., ::2]), dict(q=q.transpose(0, 1)), dict(q_out=o[:, :, :3]), dict(q=None),
                dict(q=q.cpu()), dict(q=q.half()), dict(pairing="other"), dict(scaling="other"),
                dict(pos=torch.zeros(2, 3, device="cuda", dtype=torch.int64)), dict(pos=torch.zeros(3, device="cuda", dtype=torch.int32))):
        a = dict(dict(q=q, q_out=o, pairing="half", scaling="none", pos=None), **bad)
        with pytest.raises((ValueError, TypeError)):
            L.liger_rope_scaled_fwd(a["q"], None, a["q_out"], None, 8, pos=a["pos"], pairing=a["pairing"], scaling=a["scaling"])
    for bad in (dict(rotary_dim=7), dict(rotary_dim=18), dict(scaling="yarn"), dict(theta=-1.0), dict(scaling="linear", factor=0.0)):
        with pytest.raises(L.LigerError):
            L.liger_rope_scaled_fwd(q, None, o, None, **dict(dict(rotary_dim=8), **bad))
