"""Instructions of a whole warp (".aligned") in the tensor-core products: PTX leaves it undefined what
they do in a warp whose lanes are apart, so every function that holds one first brings them together."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_efficient_optimizer_gb300", "csrc")


def functions(text):
    """{name: body} of the device functions at the top level of tc_gemm.cuh."""
    out = {}
    for m in re.finditer(r"__device__ __forceinline__ \w+ (\w+)\([^)]*(?:\([^)]*\)[^)]*)*\) \{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        out[m.group(1)] = text[m.end():at - 1]
    return out


def test_lanes_meet_before_an_instruction_of_the_whole_warp():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "tc_gemm.cuh")).read())
    with_one = {name: body for name, body in functions(text).items() if ".aligned" in body}
    assert {"tmem_load", "tmem_load64", "tmem_load16", "tmem_alloc", "tmem_free", "cluster_sync", "fewer_registers",
            "more_registers"} <= set(with_one)
    assert sum(body.count(".aligned") for body in with_one.values()) == text.count(".aligned")
    for name, body in with_one.items():
        assert body.strip().startswith("__syncwarp();"), name
    for file in ("muon.cu", "linear_ce.cu"):
        assert ".aligned" not in open(os.path.join(CSRC, file)).read()
