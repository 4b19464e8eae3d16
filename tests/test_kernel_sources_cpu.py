"""Rules of the CUDA sources that no run can show to be kept (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_decode_02_b200", "csrc")


def _kernel(file, name):
    """Text of a __global__ function, without comments."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(r"__global__[^;{]*\b%s\(" % name, text).end()
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(f"{name} has no end")


def test_verification_writes_other_ctas_memory_only_after_they_have_started():
    """A CTA's shared memory exists once the CTA runs: every thread of the cluster arrives at a
    barrier at entry and waits for it before the first store into another CTA."""
    body = _kernel("qsa_verify.cu", "verify_kernel")
    push = body.index("map_shared_rank")
    assert 0 <= body.find("cluster_arrive_relaxed();") < body.find("pdl_wait();") < push
    wait = body.find("cluster_wait();")
    assert 0 <= wait < push
    # all threads reach it: not inside a branch, no return before it
    assert body[:wait].count("{") - body[:wait].count("}") == 1 and "return" not in body[:wait]
