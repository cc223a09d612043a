"""A product of CTA pairs that gives up on a wait: the projections' launches ask for NaN in what was not finished, the epilogue of every
kind that they use writes it, and no wait of the epilogue is satisfied by products that ended early."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_rmsnorm_fwd_gb300", "csrc")


def _text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_projections_ask_for_nan_in_what_is_not_finished():
    text = _text("linear_act.cu")
    params = re.findall(r"EpiParams (\w+)\{\};", text)
    assert len(params) == text.count("launch_gemm<") - 1 == 3       # dW has two launches from one set of parameters
    for name in params:
        assert re.search(r"\b" + name + r"\.nan_unfinished = 1;", text), name
    kinds = set(re.findall(r"launch_gemm<\d, \d, (EPI_\w+)", text))
    expired = re.search(r"if \(!got\) \{(.*?)\n            \}\n", _text("tc_gemm.cuh"), re.S).group(1)
    assert "unfinished_rows(" in expired and kinds <= set(re.findall(r"EPI == (EPI_\w+)", expired))
    assert re.search(r"for \(; t < items; t \+= nunits\)", expired)     # this tile and all of the unit's after it


def test_products_that_end_early_do_not_arrive_where_the_epilogue_waits():
    text = _text("tc_gemm.cuh")
    ended = re.search(r"if \(!ok && any\) \{(.*?)\n            \}", text, re.S).group(1)
    assert re.findall(r"commit\((\w+)", ended) == ["spare_bar"] and re.findall(r"mbar_wait\((\w+)", ended) == ["spare_bar"]
    assert "mbar_init(spare_bar, 1);" in text
    # the place of the spare barrier: behind the address of the TMEM columns, inside the 256 bytes ahead of the staging buffers
    assert "slot = bar0 + 8u * (2 * Cfg::ST + 4);" in text and "spare_bar = slot + 8u;" in text
    stages = [int(n) for n in re.findall(r"constexpr int \w*ST\w*\s*=\s*(\d+)", text)] + \
        [int(n) for pair in re.findall(r"\bST = PAIR \? (\d+) : (\d+)", text) for n in pair]
    assert stages and all(8 * (2 * s + 5) + 8 <= 256 for s in stages)
