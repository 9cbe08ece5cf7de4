"""Warp-collective `.sync.aligned` instructions (tcgen05.ld, .st, their waits) have
to be executed by all 32 lanes together.  In the kernels' sources: between
such a call and the last lane-dependent branch before it in the order of
execution, a loop's previous pass included, stands a point at which the warp
comes together again."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_grouped_gemm_x32_b200", "csrc")
ALIGNED = r"\b(?:tmem_ld\d+|tmem_st\d+|tc_wait_ld|tc_wait_st)\("
JOIN = r"__syncwarp\(|__syncthreads\(|__all_sync\(|__any_sync\(|__ballot_sync\(|__shfl_\w+sync\(|warp_wait\("
# conditions that differ between the lanes of a warp
BRANCH = r"\bif \([^;{]*\b(?:lane|rv|elect_one|threadIdx)\b"
TOKEN = re.compile(f"(?P<call>{ALIGNED})|(?P<join>{JOIN})|(?P<branch>{BRANCH})|(?P<loop>\\b(?:for|while) \\()|(?P<open>{{)|(?P<close>}})")


def _tokens(src):
    """Tokens in order with their line numbers; comments blanked, declarations of the helpers left out."""
    src = re.sub(r"//[^\n]*", "", src)
    src = re.sub(r"__device__ __forceinline__[^\n]*\n?[^\n{]*", lambda m: "\n" * m.group().count("\n"), src)
    for m in TOKEN.finditer(src):
        yield m.lastgroup, src.count("\n", 0, m.start()) + 1, m.group()


def unjoined_calls(src):
    """Lines of aligned calls that a lane-dependent branch reaches without a joining point between."""
    toks, bad = list(_tokens(src)), set()

    def run(i, end, apart):
        """Executes toks[i:end] once; loops twice.  -> whether the lanes may be apart at the end."""
        while i < end:
            kind, line, _ = toks[i]
            if kind == "join":
                apart = False
            elif kind == "branch":
                apart = True
            elif kind == "call" and apart:
                bad.add(line)
            elif kind == "loop":
                j = i + 1
                while j < end and toks[j][0] in ("join", "branch"):  # in the loop's head
                    j += 1
                if j < end and toks[j][0] == "open":
                    depth, stop = 1, j + 1
                    while depth:
                        depth += {"open": 1, "close": -1}.get(toks[stop][0], 0)
                        stop += 1
                    for _ in range(2):
                        apart = run(j + 1, stop - 1, apart)
                    i = stop
                    continue
            i += 1
        return apart

    run(0, len(toks), False)
    return sorted(bad)


def test_the_search_itself():
    loop = "for (int i = 0; i < n; ++i) {\n%s  tmem_ld32(t, r);\n  tc_wait_ld();\n  if (!rv) continue;\n  f();\n}\n"
    assert unjoined_calls(loop % "") == [2, 3]
    assert unjoined_calls(loop % "  __syncwarp();\n") == []
    assert unjoined_calls("if (lane == 0) arrive();\ntc_wait_st();\n") == [2]
    assert unjoined_calls("if (lane == 0) arrive();\n__syncwarp();\ntc_wait_st();\n") == []
    assert unjoined_calls("if (any) f();\ntc_wait_st();\n") == []


@pytest.mark.parametrize("name", ["gemm.cu", "gemm_mxfp4.cu"])
def test_aligned_instructions(name):
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    assert re.search(ALIGNED, src)
    assert unjoined_calls(src) == []
