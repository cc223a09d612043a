"""What the products of CTA pairs leave after an expired wait (nothing expires here: the writing of NaN alone, tile by tile)."""
import ctypes
import glob
import os
import subprocess

import pytest
import torch

from transformer_rmsnorm_fwd_gb300 import build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def unfinished(tmp_path_factory):
    build.build()
    out = str(tmp_path_factory.mktemp("native") / "unfinished.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "unfinished.cu")
    objs = glob.glob(os.path.join(build.BUILD, "*.o"))
    p = subprocess.run([build.nvcc(), *build._flags(False), "-shared", "-Xlinker", "-Bsymbolic", "-o", out, src, *objs],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    lib = ctypes.CDLL(out)
    lib.unfinished.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                               ctypes.c_void_p]
    return lib.unfinished


@pytest.mark.parametrize("M,N", [(1, 8), (256, 256), (257, 264), (300, 1000), (2056, 2552)])
@pytest.mark.parametrize("pre", [True, False])
def test_every_output_becomes_nan_and_nothing_else(cuda_lib, unfinished, M, N, pre):
    ldo = N + 24
    out = torch.full((M + 3, ldo), 7.0, dtype=BF, device="cuda")
    kept = torch.full((M + 3, ldo), 7.0, dtype=torch.float16, device="cuda")
    rc = unfinished(None, 0, out.data_ptr(), kept.data_ptr() if pre else None, ldo, M, N, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for t, written in ((out, True), (kept, pre)):
        want = torch.zeros(M + 3, ldo, dtype=torch.bool, device="cuda")
        want[:M, :N] = written
        assert torch.equal(torch.isnan(t), want) and bool((t[~want] == 7.0).all())


@pytest.mark.parametrize("M,N", [(200, 256), (300, 264)])
def test_a_split_tiles_sums_become_nan(cuda_lib, unfinished, M, N):
    items, tiles = 3, -(-M // 256) * -(-N // 256)
    sums = torch.full((tiles * items * 256 + 1, 256), 7.0, device="cuda")
    out = torch.full((M, N), 7.0, dtype=BF, device="cuda")
    assert unfinished(sums.data_ptr(), items, out.data_ptr(), None, N, M, N, torch.cuda.current_stream().cuda_stream) == 0
    assert bool((out == 7.0).all()) and bool((sums[-1] == 7.0).all())
    for t in range(tiles):
        rows = min(256, M - t // -(-N // 256) * 256)      # those of the matrix: the join reads no others
        part = sums[t * items * 256:(t + 1) * items * 256].view(items, 256, 256)
        assert bool(torch.isnan(part[:, :rows]).all()) and bool((part[:, rows:] == 7.0).all())
