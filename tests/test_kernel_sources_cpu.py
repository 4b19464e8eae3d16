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


def test_loading_warps_wait_for_their_copies_before_they_end():
    """A CTA that ended with copies on their way would have them land in the next one's memory:
    whatever way the loading loop is left, a bounded wait for every ring slot follows it."""
    body = _kernel("qsa_paged_attend.cu", "paged_attend_kernel")
    loop = body.index("while (ld.left > 0)")
    end = body.index("return;", body.index("cp.async.mbarrier.arrive", loop))
    tail = body[body.rindex("parity ^= 1;", loop, end):end]
    wait = re.search(r"for \(int i = 0; i < STAGES; \+\+i\)\s*if \(!sm100::mbar_wait\(&sm\.full\[i\], ([^)]*)\)\) break;", tail)
    assert wait and "return" not in body[loop:end]

    # The parity it asks for is that of the slot's last fill, for every number of tiles: a fill
    # completes one phase of the slot's barrier, and a wait for parity p passes once the last
    # completed phase is p (before the first, that counts as 1).
    expr = wait.group(1).replace("i < slot ? parity ^ 1 : parity", "(parity ^ 1) if i < slot else parity")
    for stages in (2, 3, 5, 8):
        for tiles in range(4 * stages + 1):
            slot, parity, fills = 0, 1, [0] * stages
            for _ in range(tiles):
                fills[slot] += 1
                slot += 1
                if slot == stages:
                    slot, parity = 0, parity ^ 1
            for i in range(stages):
                last = (fills[i] - 1) % 2 if fills[i] else 1
                assert eval(expr, {"i": i, "slot": slot, "parity": parity}) == last
