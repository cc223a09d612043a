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
