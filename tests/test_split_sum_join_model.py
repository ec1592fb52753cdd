"""The sums of x x^T that are made in parts: what the warp that brings the last part may read.

A model of the orders that PTX gives (release and acquire at a counter, barriers of a warp, program order),
with the steps of the kernel's source in its order: of every lane's reads, which writes come before."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_efficient_optimizer_gb300", "csrc", "muon.cu")
LANES = 4


def steps():
    """The part that is written, the counter and the sum over the parts, as the source has them one after another."""
    text = open(SOURCE).read()
    body = text[text.index("bool end_gram_part("):]
    body = body[:body.index("\n}\n")]
    body = re.sub(r"//[^\n]*", "", body)
    names = {r"first\[p\.tile\.split": "write", r"__syncwarp\(": "warp", r"atom\.acq_rel": "counter",
             r"__shfl_sync\(": "shuffle", r"__ldcg\(": "read"}
    found = sorted((m.start(), name) for pattern, name in names.items() for m in re.finditer(pattern, body))
    return [name for _, name in found]


def ordered(program, warps, last):
    """Whether every lane of warp `last` reads after every lane of every warp has written.  Each lane carries the set of
    writes that come before what it does; a shuffle moves a value and orders nothing."""
    counter, ok = set(), True
    for w in [v for v in range(warps) if v != last] + [last]:
        seen = [set() for _ in range(LANES)]
        for op in program:
            if op == "write":
                for lane in range(LANES):
                    seen[lane].add((w, lane))
            elif op == "warp":
                everything = set().union(*seen)
                seen = [set(everything) for _ in range(LANES)]
            elif op == "counter":                      # lane 0: acquires what was released before, releases its own
                seen[0] |= counter
                counter |= seen[0]
            elif op == "read" and w == last:
                ok = ok and all(len(s) == warps * LANES for s in seen)
    return ok


@pytest.mark.parametrize("warps", [2, 3, 16])
def test_parts_are_read_behind_all_that_wrote_them(warps):
    program = steps()
    assert program.count("counter") == program.count("read") == program.count("write") == 1
    assert all(ordered(program, warps, last) for last in range(warps))


def test_the_model_sees_a_missing_barrier():
    whole = ["write", "warp", "counter", "warp", "shuffle", "read"]
    assert ordered(whole, 3, 1)
    for k in (1, 3):
        assert not ordered(whole[:k] + whole[k + 1:], 3, 1)
