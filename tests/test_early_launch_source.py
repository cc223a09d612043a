"""Kernels that are set up while the one before them runs read what that one may still be writing: no read-only loads."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_rmsnorm_fwd_gb300", "csrc")


def _kernels(text):
    """(name, parameters, body) of every __global__ function that is defined in the text."""
    for m in re.finditer(r"__global__", text):
        brace = text.index("{", m.start())
        if -1 < text.find(";", m.start()) < brace:
            continue
        close = text.rindex(")", m.start(), brace)
        depth, at = 0, close
        while True:
            depth += {")": 1, "(": -1}.get(text[at], 0)
            if depth == 0:
                break
            at -= 1
        end, depth = brace, 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            if depth == 0:
                break
            end += 1
        yield re.search(r"(\w+)\s*$", text[m.start():at]).group(1), text[at:close + 1], text[brace:end]


def _sources():
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(f) as h:
            yield os.path.basename(f), re.sub(r"//[^\n]*", "", h.read())


def test_kernels_launched_early_wait_and_read_by_ordinary_loads():
    waiting, found = set(), []
    for f, text in _sources():
        for name, params, body in _kernels(text):
            if "wait_for_stream()" not in body:
                continue
            waiting.add(name)
            if name == "tc_gemm_kernel":        # its fused QKV epilogue reads the bias so, and is not launched early (below)
                body = re.sub(r"__ldg\(reinterpret_cast<const float4\*>\(bh ", "", body)
            if re.search(r"const\s+[\w:]+(\s+\w+)*\s*\*\s*__restrict__", params) or re.search(r"ldg16_nc|__ldg|\.nc\.", body):
                found.append((f, name))
    assert not found, found
    assert "early" not in dict(_sources())["rmsnorm_qkv_rope.cu"]
    assert {"policy_rows_bf16", "head_gemm", "split_join", "block_norm_fwd_ring", "swiglu_bwd_ckpt8_vec", "tc_gemm_kernel"} <= waiting
    # every kernel handed to launch_early is one of them
    for f, text in _sources():
        for call in re.findall(r"launch_early\(\s*(?:\"[^\"]*\"|who)\s*,\s*([^;]*?);", text, re.S):
            for name in re.findall(r"\b(?:block_norm|swiglu|policy|logp|head|sort|label|masked|split)_\w+(?=[<,\s)])", call.split("dim3")[0]):
                if any(re.search(r"__global__[^;{]*\b" + name + r"\s*\(", t) for _, t in _sources()):
                    assert name in waiting, (f, name)
