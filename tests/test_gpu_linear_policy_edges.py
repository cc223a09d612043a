"""The policy loss and the log-probabilities where they rarely go: a GEMM that gave up on a bounded wait, tiles of the
vocabulary without a finite logit, very large vocabularies."""
import ctypes
import glob
import math
import os
import subprocess

import pytest
import torch

from test_gpu_linear_policy import IGN, L, _call, _inputs, _ref   # noqa: F401
from transformer_rmsnorm_fwd_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def compacted(L, tmp_path_factory):  # noqa: F811
    """tests/native/expired_wait.cu, linked with the library's other units."""
    build.build()
    out = str(tmp_path_factory.mktemp("native") / "expired_wait.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "expired_wait.cu")
    objs = [o for o in glob.glob(os.path.join(build.BUILD, "*.o")) if os.path.basename(o) != "linear_ce.cu.o"]
    p = subprocess.run([build.nvcc(), *build._flags(False), "-shared", "-Xlinker", "-Bsymbolic", "-o", out, src, *objs],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    lib = ctypes.CDLL(out)
    lib.policy_compacted.argtypes = ([ctypes.c_void_p] * 5 + [ctypes.c_int64] * 4 + [ctypes.c_void_p] * 6 +
                                     [ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p])
    return lib


def test_an_expired_wait_of_compacted_tokens_reaches_logp(L, compacted):  # noqa: F811
    """Where the tokens are compacted the GEMMs record an expired wait in that run's own header: logp, loss and stats are NaN."""
    T, H, V = 900, 128, 2000
    i = _inputs(T, H, V, "bf16", [0, T], seed=3, masked=0.6)
    valid = i["valid"]
    n = int(valid.sum())
    want = _call(L, i, "bf16", "token_mean", 0.2, 0.2, 0.0, 1.0, ref=False)

    def run(expired):
        ws = torch.full((L.liger_linear_policy_workspace(T, H, V),), 255, dtype=torch.uint8, device="cuda")
        o = {k: torch.full_like(v, 7.0) for k, v in want.items()}
        p = [t.data_ptr() for t in (i["X"], i["W"], i["labels"], i["old"], i["adv"])]
        q = [o[k].data_ptr() for k in ("loss", "stats", "logp", "dX", "dW")]
        rc = compacted.policy_compacted(*p, T, H, V, n, *q, ws.data_ptr(), ws.numel(), expired,
                                        torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        return o
    o = run(0)
    assert all(torch.equal(o[k], want[k]) for k in want)        # as the library's call
    o = run(1)
    assert bool(torch.isnan(o["logp"][valid]).all()) and bool((o["logp"][~valid] == 0).all())
    assert math.isnan(float(o["loss"])) and bool(torch.isnan(o["stats"]).all())


@pytest.mark.parametrize("wait", [True, False])
@pytest.mark.parametrize("T", [3, 5, 40, 300])
@pytest.mark.parametrize("V,rows", [(257, [256]), (513, [512]), (600, list(range(256, 512))), (700, list(range(512, 700)))])
def test_a_tile_of_the_vocabulary_without_a_finite_logit(L, T, V, rows, wait):  # noqa: F811
    """Rows of the head whose logits are -inf have probability 0, also where they are all there is of a tile: logp, the loss and
    the gradients are those without these rows.  Their weights are finite (-3e38 at a hidden state of 4), so that 0 times them is 0."""
    H = 64
    i = _inputs(T, H, V, "bf16", [0, T], seed=V + T, masked=0.0)
    i["X"][:, 5] = 4.0
    i["W"][:, 5] = 0.0
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[rows] = False
    i["labels"] %= 256                                  # labels in front of every such tile
    i["W"][rows] = 0.0
    i["W"][rows, 5] = -3.0e38
    few = dict(i, W=i["W"][keep])
    lp = torch.log_softmax(few["X"].double() @ few["W"].double().T, 1).gather(1, i["labels"][:, None])[:, 0]
    i["old"] = few["old"] = (lp - 0.1).float()
    i["ref"] = few["ref"] = (lp + 0.2).float()
    r = _ref(few, "token_mean", 0.2, 0.2, 0.1, 1.0)
    o = _call(L, i, "bf16", "token_mean", 0.2, 0.2, 0.1, 1.0, wait=wait)
    assert bool(((o["logp"].double() - r["logp"]).abs() <= r["eps"]).all())
    assert abs(float(o["loss"]) - r["loss"]) <= r["loss_off"] + 2 ** -22 * abs(r["loss"])
    assert bool((o["dW"][rows] == 0).all())
    assert bool(torch.isfinite(o["dW"]).all()) and bool(torch.isfinite(o["dX"]).all())
    # P and D rounded to bf16 (2^-8 each), the logits' errors, sums of at most 700 terms in fp32
    for k, got in (("dX", o["dX"]), ("dW", o["dW"][keep])):
        bound = 2.0 ** -8 * r[k].abs() + (2 * 2.0 ** -8 + 3 * r["e"] + 2.0 ** -14) * r["m" + k[1]]
        assert bool(((got.double() - r[k]).abs() <= bound).all()), k
    ws = torch.empty(L.liger_linear_logp_workspace(T, H, V), dtype=torch.uint8, device="cuda")
    logp = torch.full((T,), 7.0, device="cuda")
    L.liger_linear_logp_fwd(i["X"], i["W"], i["labels"], logp, ws, wait=wait)
    assert bool(((logp.double() - r["logp"]).abs() <= r["eps"]).all())


def test_cross_entropy_with_a_tile_without_a_finite_logit(L):  # noqa: F811
    """The cross-entropies share the logits' epilogue."""
    T, H, V = 40, 64, 513
    i = _inputs(T, H, V, "bf16", [0, T], seed=1, masked=0.0)
    i["X"][:, 5], i["W"][:, 5], i["W"][512] = 4.0, 0.0, 0.0
    i["W"][512, 5] = -3.0e38
    i["labels"] %= 256
    lp = torch.log_softmax(i["X"].double() @ i["W"][:512].double().T, 1).gather(1, i["labels"][:, None])[:, 0]
    loss, dX, dW = torch.zeros(1, device="cuda"), torch.empty_like(i["X"]), torch.empty_like(i["W"])
    for ws, fn in ((L.liger_linear_ce_workspace(T, H, V), L.liger_linear_ce_fwd_bwd),
                   (L.liger_linear_ce_two_pass_workspace(T, H, V), L.liger_linear_ce_two_pass_fwd_bwd)):
        fn(i["X"], i["W"], i["labels"], loss, dX, dW, torch.empty(ws, dtype=torch.uint8, device="cuda"))
        xw = float((i["X"].abs().double() @ i["W"][:512].abs().double().T).max())
        assert abs(float(loss) + float(lp.mean())) <= (2 * 64 + 64) * 2.0 ** -23 * xw
        assert bool((dW[512] == 0).all()) and bool(torch.isfinite(dX).all())


def test_a_vocabulary_of_millions(L):  # noqa: F811
    """A row's tiles number more than shared memory would hold factors for; every piece of the row keeps its own only."""
    T, H, V = 2, 64, 3_200_003
    i = _inputs(T, H, V, "bf16", [0, T], seed=6, masked=0.0)
    r = _ref(i, "token_mean", 0.2, 0.2, 0.1, 1.0)
    o = _call(L, i, "bf16", "token_mean", 0.2, 0.2, 0.1, 1.0)
    assert bool(((o["logp"].double() - r["logp"]).abs() <= r["eps"]).all())
    assert abs(float(o["loss"]) - r["loss"]) <= r["loss_off"] + 2 ** -22 * abs(r["loss"])
    for k in ("dX", "dW"):      # sums over V / 16 steps of the tensor cores in 76 runs
        bound = 2.0 ** -8 * r[k].abs() + (2 * 2.0 ** -8 + 3 * r["e"] + 2.0 ** -10) * r["m" + k[1]]
        assert bool(((o[k].double() - r[k]).abs() <= bound).all()), k
