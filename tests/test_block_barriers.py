"""Barriers of a block in kernels whose warps take different instantiations of one function, read from the source
(no GPU): such warps may not meet at __syncthreads(), which all threads of the block have to reach at the same place."""
import os
import re

import top_group_sparse_gb300

CSRC = os.path.join(os.path.dirname(top_group_sparse_gb300.__file__), "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_the_steps_of_new_tokens_meet_at_a_barrier_with_a_count():
    code = _code("append.cu")
    # one CTA's warps go into both families
    assert re.search(r"if \(step < a\.family\[0\]\.steps\) append_step<T, D, DI, 0>\(.*?\);\s*else append_step<T, D, DI, 1>\(", code, flags=re.S)
    assert "__syncthreads" not in code
    barriers = re.findall(r'"(bar(?:rier)?[.\w]*)\s+([^;"]*);"\s*::"r"\(([^)]*)\)', code)
    assert barriers == [("barrier.cta.sync", "1, %0", "blockDim.x")]
    step = code[code.index("void append_step("):code.index("append_kernel(const")]
    assert step.count("meet_all_steps();") == 2     # before the rounds, and once in each
    loop = re.search(r"while \(([^)]*)\) \{", step).group(1)
    assert loop == "first < a.batch"                # of neither family: the rounds are the same
