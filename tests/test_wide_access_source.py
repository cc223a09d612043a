"""Arrays in registers or shared memory that are read or written several elements at a time say that they are aligned for it:
the language gives an array the alignment of its element only."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_rmsnorm_fwd_gb300", "csrc")
WIDE = {"uint2": 8, "float2": 8, "uint4": 16, "float4": 16}
DECLARED = re.compile(r"^\s*((?:extern\s+)?(?:__shared__\s+)?)(?:(?:__align__|alignas)\((\d+)\)\s+)?"
                      r"(?:float|__half|__nv_bfloat16|uint8_t|uint16_t|uint32_t|int)\s+(\w+\s*\[[^;=()]*(?:\([^;=()]*\)[^;=()]*)*(?:=[^;]*)?);")
CAST = re.compile(r"reinterpret_cast<\s*(?:const\s+)?(uint2|uint4|float2|float4)\s*\*\s*>\(\s*&?\s*(\w+)")


def _sources():
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(f) as h:
            yield os.path.basename(f), [re.sub(r"//.*", "", line) for line in h]


def test_arrays_that_are_accessed_wide_are_aligned():
    found, seen = [], 0
    for f, lines in _sources():
        arrays = {}     # name -> alignment of the latest declaration above
        for n, line in enumerate(lines, 1):
            if line.startswith("}"):
                arrays = {}
            d = DECLARED.match(line)
            if d:
                for name in re.findall(r"(\w+)\s*\[", d.group(3)):
                    arrays[name] = int(d.group(2) or 0)
            for kind, name in CAST.findall(line):
                if name in arrays:
                    seen += 1
                    if arrays[name] < WIDE[kind]:
                        found.append((f, n, name))
    assert not found, found
    assert seen >= 10       # the pattern still finds the accesses


def test_keys_of_a_scored_row_are_aligned_for_pairs():
    """Loops over the 8-byte keys of a block may be read in pairs."""
    text = dict((f, "".join(lines)) for f, lines in _sources())["token_logp.cu"]
    body = re.search(r"struct (alignas\(16\) )?RowShared \{(.*?)\};", text, re.S)
    assert body.group(1)
    for name in ("best", "groups", "red"):
        assert re.search(r"alignas\(16\) unsigned long long " + name + r"\[", body.group(2)), name
    assert re.search(r"extern __shared__ __align__\(16\) unsigned long long list\[\]", text)
